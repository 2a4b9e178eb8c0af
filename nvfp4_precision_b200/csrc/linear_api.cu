// C ABI of the linear layers in NVFP4 and of the gated norms: argument
// validation, workspace layout and launches on the caller's stream.  See
// include/fp4attn.h for the contract of each entry point.
#include <cstdint>

#include "fp4attn.h"
#include "kernels.h"
#include "nvfp4_rows.cuh"

namespace fp4attn {

namespace {

constexpr int64_t kMaxRows = 4194304;  // 2^22: tile counts and coordinates stay far inside 32 bits
constexpr int64_t kMaxK = 1048576;
constexpr int64_t kMaxStride = (int64_t)1 << 39;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool good(const void* p) { return p && aligned16(p); }

int check_rows(int64_t rows) {
    if (rows < 0) return FP4ATTN_ERR_INVALID_ARG;
    return rows > kMaxRows ? FP4ATTN_ERR_UNSUPPORTED : FP4ATTN_OK;
}
int check_k(int64_t K) {
    if (K <= 0) return FP4ATTN_ERR_INVALID_ARG;
    return (K % 32 || K > kMaxK) ? FP4ATTN_ERR_UNSUPPORTED : FP4ATTN_OK;
}
int check_mnk(int64_t M, int64_t N, int64_t K) {
    int st = check_rows(M);
    if (st == FP4ATTN_OK) st = check_rows(N);
    if (st == FP4ATTN_OK) st = check_k(K);
    return st;
}

int launch_status(cudaError_t e) {
    if (e == cudaSuccess) return FP4ATTN_OK;
    (void)cudaGetLastError();
    return FP4ATTN_ERR_CUDA;
}
int clear_error(int st) {
    if (st != FP4ATTN_OK) (void)cudaGetLastError();
    return st;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

}  // namespace fp4attn

using namespace fp4attn;

extern "C" {

size_t fp4attn_scale_tile_bytes(int64_t rows, int64_t K) {
    if (check_rows(rows) != FP4ATTN_OK || check_k(K) != FP4ATTN_OK) return 0;
    return (size_t)scale_tile_bytes(rows, K);
}

size_t fp4attn_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    (void)N;  // the product itself needs none
    const size_t base = lws_codes_offset();
    if (check_rows(M) != FP4ATTN_OK || check_k(K) != FP4ATTN_OK) return base;
    return base + round256((size_t)(M * (K / 2))) + round256((size_t)scale_tile_bytes(M, K));
}

int fp4attn_quantize_rows(const void* x, int x_type, int64_t x_stride, int64_t rows, int64_t K, float* gscale,
                          uint32_t flags, uint8_t* codes, uint8_t* scales, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
    int st = check_rows(rows);
    if (st == FP4ATTN_OK) st = check_k(K);
    if (st != FP4ATTN_OK) return st;
    if (x_type != FP4ATTN_BF16 && x_type != FP4ATTN_F32) return FP4ATTN_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)FP4ATTN_DYNAMIC_GSCALE) return FP4ATTN_ERR_INVALID_ARG;
    const bool dynamic = (flags & FP4ATTN_DYNAMIC_GSCALE) != 0;
    if ((dynamic && !gscale) || !aligned4(gscale)) return FP4ATTN_ERR_INVALID_ARG;
    if (!good(workspace) || workspace_bytes < lws_codes_offset()) return FP4ATTN_ERR_WORKSPACE;
    if (rows == 0) return dynamic ? launch_status(launch_store_gscales(gscale, gscale, stream)) : FP4ATTN_OK;
    const int64_t unit = x_type == FP4ATTN_F32 ? 4 : 8;
    if (rows > 1 && (x_stride < K || x_stride % unit || x_stride >= kMaxStride)) return FP4ATTN_ERR_INVALID_ARG;
    if (!good(x) || !good(codes) || !good(scales)) return FP4ATTN_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    QuantRowsArgs a{};
    a.x = x;
    a.ld = rows > 1 ? x_stride : K;
    a.rows = rows;
    a.K = K;
    a.g = dynamic ? nullptr : gscale;
    a.g_out = dynamic ? gscale : nullptr;
    a.dynamic = dynamic;
    a.part = reinterpret_cast<float*>(ws + lws_part_offset());
    a.codes = codes;
    a.scales = scales;
    a.status = reinterpret_cast<int*>(ws);
    return launch_status(launch_quantize_rows(a, x_type == FP4ATTN_F32, stream));
}

int fp4attn_dequant_rows(const uint8_t* codes, const uint8_t* scales, const float* gscale, int64_t rows, int64_t K,
                         void* out, int out_type, cudaStream_t stream) {
    int st = check_rows(rows);
    if (st == FP4ATTN_OK) st = check_k(K);
    if (st != FP4ATTN_OK) return st;
    if (out_type != FP4ATTN_BF16 && out_type != FP4ATTN_F32) return FP4ATTN_ERR_INVALID_ARG;
    if (!aligned4(gscale)) return FP4ATTN_ERR_INVALID_ARG;
    if (rows == 0) return FP4ATTN_OK;
    if (!good(codes) || !good(scales) || !good(out)) return FP4ATTN_ERR_INVALID_ARG;
    return launch_status(launch_dequant_rows(codes, scales, gscale, rows, K, out, out_type == FP4ATTN_F32, stream));
}

int fp4attn_gemm(const uint8_t* x_codes, const uint8_t* x_scales, const float* gx, const uint8_t* w_codes,
                 const uint8_t* w_scales, const float* gw, const void* bias, int64_t M, int64_t N, int64_t K, void* y,
                 int64_t y_stride, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_mnk(M, N, K);
    if (st != FP4ATTN_OK) return st;
    if (!good(workspace) || workspace_bytes < lws_codes_offset()) return FP4ATTN_ERR_WORKSPACE;
    if (!aligned4(gx) || !aligned4(gw)) return FP4ATTN_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return FP4ATTN_OK;
    if (!good(x_codes) || !good(x_scales) || !good(w_codes) || !good(w_scales) || !good(y) || !aligned16(bias))
        return FP4ATTN_ERR_INVALID_ARG;
    if (M > 1 && (y_stride < N || y_stride >= kMaxStride)) return FP4ATTN_ERR_INVALID_ARG;
    GemmFp4Args a{};
    a.x_codes = x_codes;
    a.x_scales = x_scales;
    a.gx = gx;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.gw = gw;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<__nv_bfloat16*>(y);
    a.ld = M > 1 ? y_stride : N;
    a.status = static_cast<int*>(workspace);
    return clear_error(launch_gemm_fp4(a, stream));
}

int fp4attn_linear(const void* x, int64_t x_stride, float* gx, uint32_t flags, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gw, const void* bias, int64_t M, int64_t N, int64_t K,
                   void* y, int64_t y_stride, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_mnk(M, N, K);
    if (st != FP4ATTN_OK) return st;
    if (flags & ~(uint32_t)FP4ATTN_DYNAMIC_GSCALE) return FP4ATTN_ERR_INVALID_ARG;
    const bool dynamic = (flags & FP4ATTN_DYNAMIC_GSCALE) != 0;
    if (!good(workspace) || workspace_bytes < fp4attn_linear_workspace_bytes(M, N, K)) return FP4ATTN_ERR_WORKSPACE;
    if (!aligned4(gx) || !aligned4(gw)) return FP4ATTN_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {
        // no product; a computed scale is still written where the caller asked for it
        if (!dynamic || !gx) return FP4ATTN_OK;
        if (M == 0) return launch_status(launch_store_gscales(gx, gx, stream));
    }
    if (!good(x) || !aligned16(bias)) return FP4ATTN_ERR_INVALID_ARG;
    if (N > 0 && (!good(w_codes) || !good(w_scales) || !good(y))) return FP4ATTN_ERR_INVALID_ARG;
    if (M > 1 && (x_stride < K || x_stride % 8 || x_stride >= kMaxStride || y_stride < N || y_stride >= kMaxStride))
        return FP4ATTN_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* g = dynamic && !gx ? reinterpret_cast<float*>(ws + WS_GSCALE_OFFSET) : gx;
    QuantRowsArgs q{};
    q.x = x;
    q.ld = M > 1 ? x_stride : K;
    q.rows = M;
    q.K = K;
    q.g = dynamic ? nullptr : g;
    q.g_out = dynamic ? g : nullptr;
    q.dynamic = dynamic;
    q.pdl = true;
    q.part = reinterpret_cast<float*>(ws + lws_part_offset());
    q.codes = ws + lws_codes_offset();
    q.scales = q.codes + round256((size_t)(M * (K / 2)));
    q.status = reinterpret_cast<int*>(ws);
    st = launch_status(launch_quantize_rows(q, false, stream));
    if (st != FP4ATTN_OK || N == 0) return st;
    GemmFp4Args a{};
    a.x_codes = q.codes;
    a.x_scales = q.scales;
    a.gx = g;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.gw = gw;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<__nv_bfloat16*>(y);
    a.ld = M > 1 ? y_stride : N;
    a.after_quantize = true;
    a.status = q.status;
    return clear_error(launch_gemm_fp4(a, stream));
}

}  // extern "C"
