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
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // bytes stay below what tensor maps hold

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

// Workspace of the linear layer's backward: [0,256) status word and spare; W~
// and X~ in bf16; partial column sums of dy; parts of split tiles.
size_t lbws_x_offset(int64_t N, int64_t K) { return WS_STATUS_BYTES + round256((size_t)(N * K) * 2); }
size_t lbws_colsum_offset(int64_t M, int64_t N, int64_t K) { return lbws_x_offset(N, K) + round256((size_t)(M * K) * 2); }
size_t lbws_part_offset(int64_t M, int64_t N, int64_t K) {
    return lbws_colsum_offset(M, N, K) + round256((size_t)N * COLSUM_PARTS * 4);
}

constexpr int64_t kMaxC = 16384;
constexpr int64_t kMaxGroups = 1048576;

int check_norm_sizes(int64_t rows, int64_t C, int64_t groups) {
    // no rows: any number of samples, none too
    if (rows < 0 || C <= 0 || groups < 0 || (rows > 0 && (groups == 0 || rows % groups))) return FP4ATTN_ERR_INVALID_ARG;
    return (rows > kMaxRows || C % 8 || C > kMaxC || groups > kMaxGroups) ? FP4ATTN_ERR_UNSUPPORTED : FP4ATTN_OK;
}
// A row matrix: 16-byte aligned, rows a multiple of `unit` elements apart.
bool bad_rows(const void* p, int64_t ld, int64_t rows, int64_t C, int64_t unit) {
    return !aligned16(p) || (rows > 1 && (ld < C || ld % unit || ld >= kMaxStride));
}
bool bad_vector(const void* p, int64_t ld, int64_t groups, int64_t C) {
    return !aligned16(p) || (p && groups > 1 && (ld < C || ld % 8 || ld >= kMaxStride));
}
int check_norm_vectors(const fp4attn_norm_vectors& v, int64_t groups, int64_t C) {
    return (!aligned16(v.post_weight) || !aligned16(v.pre_weight) || bad_vector(v.gate, v.gate_stride, groups, C) ||
            bad_vector(v.scale, v.scale_stride, groups, C) || bad_vector(v.shift, v.shift_stride, groups, C))
               ? FP4ATTN_ERR_INVALID_ARG
               : FP4ATTN_OK;
}

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
    a.weight_ready = true;
    a.status = q.status;
    return clear_error(launch_gemm_fp4(a, stream));
}

size_t fp4attn_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_mnk(M, N, K) != FP4ATTN_OK) return WS_STATUS_BYTES;
    // for any choice of gradients
    size_t parts = 0;
    for (int want = 1; want < 4; ++want) {
        const size_t b = linear_backward_part_bytes(linear_backward_plan(M, N, K, want & 1, want & 2));
        parts = b > parts ? b : parts;
    }
    return lbws_part_offset(M, N, K) + round256(parts);
}

int fp4attn_linear_backward(const void* dy, int64_t dy_stride, const uint8_t* x_codes, const uint8_t* x_scales,
                            const float* gx, const uint8_t* w_codes, const uint8_t* w_scales, const float* gw, int64_t M,
                            int64_t N, int64_t K, void* dx, int64_t dx_stride, void* dw, float* dbias, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
    const int st = check_mnk(M, N, K);
    if (st != FP4ATTN_OK) return st;
    const LinearBwdPlan plan = linear_backward_plan(M, N, K, dw != nullptr, dx != nullptr);
    if (!good(workspace) || workspace_bytes < lbws_part_offset(M, N, K) + round256(linear_backward_part_bytes(plan)))
        return FP4ATTN_ERR_WORKSPACE;
    if (!aligned4(gx) || !aligned4(gw) || !aligned4(dbias)) return FP4ATTN_ERR_INVALID_ARG;
    if (dx && M > 0 && bad_rows(dx, dx_stride, M, K, 8)) return FP4ATTN_ERR_INVALID_ARG;
    if (!aligned16(dw)) return FP4ATTN_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {
        // sums over nothing
        cudaError_t e = cudaSuccess;
        if (dx && M > 0)
            e = cudaMemset2DAsync(dx, (size_t)(M > 1 ? dx_stride : K) * 2, 0, (size_t)K * 2, (size_t)M, stream);
        if (e == cudaSuccess && dw && N > 0) e = cudaMemsetAsync(dw, 0, (size_t)(N * K) * 2, stream);
        if (e == cudaSuccess && dbias && N > 0) e = cudaMemsetAsync(dbias, 0, (size_t)N * 4, stream);
        return launch_status(e);
    }
    if (!dy || bad_rows(dy, dy_stride, M, N, 8)) return FP4ATTN_ERR_INVALID_ARG;
    if (dx && (!good(w_codes) || !good(w_scales))) return FP4ATTN_ERR_INVALID_ARG;
    if (dw && (!good(x_codes) || !good(x_scales))) return FP4ATTN_ERR_INVALID_ARG;
    if (!dx && !dw && !dbias) return FP4ATTN_OK;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    LinearBwdArgs a{};
    a.dy = static_cast<const __nv_bfloat16*>(dy);
    a.ld_dy = M > 1 ? dy_stride : (N + 7) / 8 * 8;
    a.x_codes = x_codes;
    a.x_scales = x_scales;
    a.gx = gx;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.gw = gw;
    a.M = M;
    a.N = N;
    a.K = K;
    a.dx = static_cast<__nv_bfloat16*>(dx);
    a.ld_dx = M > 1 ? dx_stride : K;
    a.dw = static_cast<__nv_bfloat16*>(dw);
    a.dbias = dbias;
    a.w_bf16 = reinterpret_cast<__nv_bfloat16*>(ws + WS_STATUS_BYTES);
    a.x_bf16 = reinterpret_cast<__nv_bfloat16*>(ws + lbws_x_offset(N, K));
    a.colsum_part = reinterpret_cast<float*>(ws + lbws_colsum_offset(M, N, K));
    a.part = reinterpret_cast<float*>(ws + lbws_part_offset(M, N, K));
    a.plan = plan;
    a.status = static_cast<int*>(workspace);
    return clear_error(launch_linear_backward(a, stream));
}

int fp4attn_norm_gate(const void* x, int x_type, int64_t x_stride, const void* h, int64_t h_stride,
                      const fp4attn_norm_vectors* vectors, int64_t rows, int64_t C, int64_t groups, float eps,
                      uint32_t flags, void* y, int64_t y_stride, void* z, int64_t z_stride, uint8_t* z_codes,
                      uint8_t* z_scales, const float* z_gscale, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
    int st = check_norm_sizes(rows, C, groups);
    if (st != FP4ATTN_OK) return st;
    const bool quant = z_codes || z_scales;
    if (!vectors || (x_type != FP4ATTN_BF16 && x_type != FP4ATTN_F32) || (flags & ~(uint32_t)FP4ATTN_LAYER_NORM) ||
        !(eps >= 0.0f && eps <= 3.0e38f))
        return FP4ATTN_ERR_INVALID_ARG;
    if (quant && (!z_codes || !z_scales || z || !aligned4(z_gscale))) return FP4ATTN_ERR_INVALID_ARG;
    if (quant && C % 32) return FP4ATTN_ERR_UNSUPPORTED;
    if (workspace ? (!good(workspace) || workspace_bytes < lws_codes_offset()) : quant) return FP4ATTN_ERR_WORKSPACE;
    if (rows == 0) return FP4ATTN_OK;
    st = check_norm_vectors(*vectors, groups, C);
    if (st != FP4ATTN_OK) return st;
    const int64_t unit = x_type == FP4ATTN_F32 ? 4 : 8;
    if (!x || (!y && !z && !quant) || bad_rows(x, x_stride, rows, C, unit) || bad_rows(h, h ? h_stride : C, rows, C, 8) ||
        bad_rows(y, y ? y_stride : C, rows, C, unit) || bad_rows(z, z ? z_stride : C, rows, C, 8) ||
        !aligned16(z_codes) || !aligned16(z_scales))
        return FP4ATTN_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x;
    a.ldx = x_stride;
    a.h = static_cast<const __nv_bfloat16*>(h);
    a.ldh = h_stride;
    a.post = static_cast<const __nv_bfloat16*>(vectors->post_weight);
    a.gate = static_cast<const __nv_bfloat16*>(vectors->gate);
    a.pre = static_cast<const __nv_bfloat16*>(vectors->pre_weight);
    a.scale = static_cast<const __nv_bfloat16*>(vectors->scale);
    a.shift = static_cast<const __nv_bfloat16*>(vectors->shift);
    a.lgate = vectors->gate_stride;
    a.lscale = vectors->scale_stride;
    a.lshift = vectors->shift_stride;
    a.rows = rows;
    a.rows_per_group = rows / groups;
    a.C = (int)C;
    a.eps = eps;
    a.layer = (flags & FP4ATTN_LAYER_NORM) != 0;
    a.y = y;
    a.ldy = y_stride;
    a.z = static_cast<__nv_bfloat16*>(z);
    a.ldz = z_stride;
    a.codes = z_codes;
    a.scales = z_scales;
    a.gz = z_gscale;
    a.chunks = scale_chunks(C);
    a.status = static_cast<int*>(workspace);
    return clear_error(launch_norm_gate(a, x_type == FP4ATTN_F32, stream));
}

size_t fp4attn_norm_gate_backward_workspace_bytes(int64_t rows, int64_t C, int64_t groups) {
    if (check_norm_sizes(rows, C, groups) != FP4ATTN_OK) return WS_STATUS_BYTES;
    return WS_STATUS_BYTES + round256((size_t)(groups * norm_backward_parts(rows, C, groups)) * 3 * (size_t)C * 4);
}

int fp4attn_norm_gate_backward(const void* dz, int64_t dz_stride, const void* dy, int64_t dy_stride, const void* y,
                               int64_t y_stride, int y_type, const void* h, int64_t h_stride,
                               const fp4attn_norm_vectors* vectors, int64_t rows, int64_t C, int64_t groups, float eps,
                               uint32_t flags, void* dx, int64_t dx_stride, void* dh, int64_t dh_stride, float* dshift,
                               float* dscale, float* dgate, float* dpre_weight, float* dpost_weight, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    int st = check_norm_sizes(rows, C, groups);
    if (st != FP4ATTN_OK) return st;
    if (!vectors || (y_type != FP4ATTN_BF16 && y_type != FP4ATTN_F32) || (flags & ~(uint32_t)FP4ATTN_LAYER_NORM) ||
        !(eps >= 0.0f && eps <= 3.0e38f))
        return FP4ATTN_ERR_INVALID_ARG;
    if (!good(workspace) || workspace_bytes < fp4attn_norm_gate_backward_workspace_bytes(rows, C, groups))
        return FP4ATTN_ERR_WORKSPACE;
    if (!aligned4(dshift) || !aligned4(dscale) || !aligned4(dgate) || !aligned4(dpre_weight) || !aligned4(dpost_weight))
        return FP4ATTN_ERR_INVALID_ARG;
    if (!h && (rows > 0 && (dh || dgate || dpost_weight))) return FP4ATTN_ERR_INVALID_ARG;
    if (rows == 0) {
        float* const per_group[3] = {dshift, dscale, dgate};
        float* const weights[2] = {dpre_weight, dpost_weight};
        cudaError_t e = cudaSuccess;
        for (float* p : per_group)
            if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)(groups * C) * 4, stream);
        for (float* p : weights)
            if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)C * 4, stream);
        return launch_status(e);
    }
    st = check_norm_vectors(*vectors, groups, C);
    if (st != FP4ATTN_OK) return st;
    const int64_t unit = y_type == FP4ATTN_F32 ? 4 : 8;
    if (!dz || !y || !dx || (h && !dh) || bad_rows(dz, dz_stride, rows, C, 8) || bad_rows(dy, dy ? dy_stride : C, rows, C, unit) ||
        bad_rows(y, y_stride, rows, C, unit) || bad_rows(h, h ? h_stride : C, rows, C, 8) ||
        bad_rows(dx, dx_stride, rows, C, unit) || bad_rows(dh, dh ? dh_stride : C, rows, C, 8))
        return FP4ATTN_ERR_INVALID_ARG;
    NormBwdArgs a{};
    a.dz = static_cast<const __nv_bfloat16*>(dz);
    a.lddz = dz_stride;
    a.dy = dy;
    a.lddy = dy_stride;
    a.y = y;
    a.ldy = y_stride;
    a.h = static_cast<const __nv_bfloat16*>(h);
    a.ldh = h_stride;
    a.post = static_cast<const __nv_bfloat16*>(vectors->post_weight);
    a.gate = static_cast<const __nv_bfloat16*>(vectors->gate);
    a.pre = static_cast<const __nv_bfloat16*>(vectors->pre_weight);
    a.scale = static_cast<const __nv_bfloat16*>(vectors->scale);
    a.lgate = vectors->gate_stride;
    a.lscale = vectors->scale_stride;
    a.rows = rows;
    a.rows_per_group = rows / groups;
    a.groups = groups;
    a.parts = norm_backward_parts(rows, C, groups);
    a.C = (int)C;
    a.eps = eps;
    a.layer = (flags & FP4ATTN_LAYER_NORM) != 0;
    a.dx = dx;
    a.lddx = dx_stride;
    a.dh = static_cast<__nv_bfloat16*>(dh);
    a.lddh = dh_stride;
    a.dshift = dshift;
    a.dscale = dscale;
    a.dgate = dgate;
    a.dpre = dpre_weight;
    a.dpost = dpost_weight;
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + WS_STATUS_BYTES);
    a.status = static_cast<int*>(workspace);
    return clear_error(launch_norm_gate_backward(a, y_type == FP4ATTN_F32, stream));
}

}  // extern "C"
