// NVFP4 rows: quantisation of bf16 or fp32 rows (codes, tiled scales, an
// optional computed per-tensor scale), reading them back, and column sums.
//
//   s = E4M3(amax_16 / 6 / g),  code = E2M1(v * (1 / (g s))),  value = g s code
//
// FastVideo "Pika H3 Flex in FastVideo", section "NVFP4 QAD": weights and
// activations of the linear layers in NVFP4 (one 8-bit scale per 16 values, a
// per-tensor scale).  Everything here is bound by HBM: a quantised bf16 value
// costs 2 bytes read and 9/16 written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nvfp4_rows.cuh"

namespace fp4attn {

namespace {

// One CTA covers 128 rows x 256 channels: 16 threads per row (one 16-value
// block each), 16 rows per pass, 8 passes.  A row's segment is 512 contiguous
// bytes of bf16, and the CTA's scales are four whole tiles, which meet in
// shared memory and leave as one contiguous run of 2 KB: written one by one
// they would touch a 32-byte sector per word.
constexpr int TILE_ROWS = 128, TILE_COLS = 256, QTHREADS = 256;

template <bool F32>
struct Block16 {
    uint4 w[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void* p) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) w[i] = __ldg(q + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&lo)[8], float (&hi)[8]) const {
        if constexpr (F32) {
            const uint4 a = w[0], b = w[1], c = w[2], d = w[3];
            const uint32_t x[16] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] = __uint_as_float(x[i]);
                hi[i] = __uint_as_float(x[8 + i]);
            }
        } else {
            const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[2 * i] = bf16lo(x[i]);
                lo[2 * i + 1] = bf16hi(x[i]);
                hi[2 * i] = bf16lo(x[4 + i]);
                hi[2 * i + 1] = bf16hi(x[4 + i]);
            }
        }
    }
};

__device__ __forceinline__ float amax16(const float (&lo)[8], const float (&hi)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, max_nan(fabsf(lo[i]), fabsf(hi[i])));
    return m;
}

// Largest of a value per thread over the CTA, NaN kept, in every thread.
__device__ __forceinline__ float block_max_nan(float m, float* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = m;
    __syncthreads();
    m = scratch[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) m = max_nan(m, scratch[i]);
    __syncthreads();
    return m;
}

// Largest magnitude of a row segment per CTA.  The maxima go to a list, not to
// one word by atomics: the list needs no clearing before the call.
template <bool F32>
__global__ void __launch_bounds__(QTHREADS) rows_amax_kernel(const void* x, int64_t ld, int64_t rows, int64_t K,
                                                             float* part) {
    __shared__ float scratch[QTHREADS / 32];
    const int64_t per_row = K / 16, total = rows * per_row;
    const int64_t stride = (int64_t)gridDim.x * QTHREADS;
    const char* base = static_cast<const char*>(x);
    constexpr int ES = F32 ? 4 : 2;
    float m = 0.0f;
    int64_t i = (int64_t)blockIdx.x * QTHREADS + threadIdx.x;
    int64_t r = i / per_row, c = i - r * per_row;
    const int64_t dr = stride / per_row, dc = stride - dr * per_row;
    for (; i < total; i += 4 * stride) {
        Block16<F32> b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i + u * stride < total)
                b[u].load(base + (r * ld + c * 16) * ES);
            else
                b[u].zero();
            r += dr;
            c += dc;
            if (c >= per_row) {
                c -= per_row;
                ++r;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float lo[8], hi[8];
            b[u].values(lo, hi);
            m = max_nan(m, amax16(lo, hi));
        }
    }
    m = block_max_nan(m, scratch);
    if (threadIdx.x == 0) part[blockIdx.x] = m;
}

template <bool F32>
__global__ void __launch_bounds__(QTHREADS) quantize_rows_kernel(QuantRowsArgs a) {
    __shared__ __align__(16) uint32_t tile[4 * 128];
    __shared__ float scratch[QTHREADS / 32];
    if (a.pdl) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int ES = F32 ? 4 : 2;
    const int t = threadIdx.x;
    const char* base = static_cast<const char*>(a.x);
    float g = 1.0f;
    if (a.dynamic) {
        // the maxima of the launch before, or (small inputs) all of x
        float m = 0.0f;
        if (a.n_part > 0) {
            for (int i = t; i < a.n_part; i += QTHREADS) m = max_nan(m, __ldcg(a.part + i));
        } else {
            const int64_t per_row = a.K / 16;
            for (int64_t i = t; i < a.rows * per_row; i += QTHREADS) {
                const int64_t r = i / per_row, c = i - r * per_row;
                Block16<F32> b;
                b.load(base + (r * a.ld + c * 16) * ES);
                float lo[8], hi[8];
                b.values(lo, hi);
                m = max_nan(m, amax16(lo, hi));
            }
        }
        g = computed_gscale(block_max_nan(m, scratch));
        if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) *a.g_out = g;
    } else if (a.g) {
        g = __ldg(a.g);
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0 && bad_gscale(g)) raise_status(a.status, FP4ATTN_ERR_RANGE);
    // the last row blocks first: after a pass for the maxima they are the ones still in L2
    const int64_t rb = (int64_t)gridDim.y - 1 - blockIdx.y;
    const int64_t row0 = rb * TILE_ROWS, col0 = (int64_t)blockIdx.x * TILE_COLS;
    const int blk = t & 15, rsub = t >> 4;
    const int64_t col = col0 + 16 * blk;
    const bool in_cols = col < a.K;
    bool finite = true;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Block16<F32> b[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t row = row0 + rsub + 16 * (4 * half + p);
            if (in_cols && row < a.rows)
                b[p].load(base + (row * a.ld + col) * ES);
            else
                b[p].zero();
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int rr = rsub + 16 * (4 * half + p);
            const int64_t row = row0 + rr;
            float lo[8], hi[8];
            b[p].values(lo, hi);
            const float m = amax16(lo, hi);
            finite = finite && (m < INFINITY);
            uint32_t s;
            float inv;
            row_block_scale(m, g, s, inv);
            const uint32_t c0 = row_codes8(lo, inv), c1 = row_codes8(hi, inv);
            if (in_cols && row < a.rows && FP4ATTN_IN_BOUNDS(row * (a.K / 2) + col / 2 + 8 <= a.rows * (a.K / 2), a.status))
                *reinterpret_cast<uint2*>(a.codes + row * (a.K / 2) + col / 2) = make_uint2(c0, c1);
            // four blocks of a row make a word of a tile
            uint32_t w = s << (8 * (blk & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, 1);
            w |= __shfl_xor_sync(0xffffffffu, w, 2);
            if ((blk & 3) == 0) tile[128 * (blk >> 2) + scale_word_in_tile((uint32_t)rr)] = w;
        }
    }
    if (!finite) raise_status(a.status, FP4ATTN_ERR_RANGE);
    __syncthreads();
    const int64_t chunks = scale_chunks(a.K), c0 = col0 / 64;
    const int n_tiles = (int)(chunks - c0 < 4 ? chunks - c0 : 4);
    if (t < 32 * n_tiles) {
        const int64_t off = (rb * chunks + c0) * 512 + 16 * t;
        if (FP4ATTN_IN_BOUNDS(off + 16 <= scale_tile_bytes(a.rows, a.K), a.status))
            *reinterpret_cast<uint4*>(a.scales + off) = reinterpret_cast<const uint4*>(tile)[t];
    }
}

// The values of quantised rows: fl(fl(g s) * e2m1), to fp32 or rounded to bf16
// (exact in bf16 for g a power of two).  Same tiling as the quantiser.
template <bool F32>
__global__ void __launch_bounds__(QTHREADS) dequant_rows_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, const float* gp,
                                                                int64_t rows, int64_t K, void* out) {
    __shared__ __align__(16) uint32_t tile[4 * 128];
    const int t = threadIdx.x;
    const int64_t rb = blockIdx.y, row0 = rb * TILE_ROWS, col0 = (int64_t)blockIdx.x * TILE_COLS;
    const int64_t chunks = scale_chunks(K), ch0 = col0 / 64;
    const int n_tiles = (int)(chunks - ch0 < 4 ? chunks - ch0 : 4);
    if (t < 32 * n_tiles)
        reinterpret_cast<uint4*>(tile)[t] =
            __ldg(reinterpret_cast<const uint4*>(scales + (rb * chunks + ch0) * 512 + 16 * t));
    const float g = gp ? __ldg(gp) : 1.0f;
    const int blk = t & 15, rsub = t >> 4;
    const int64_t col = col0 + 16 * blk;
    __syncthreads();
    if (col >= K) return;
    uint2 c[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t row = row0 + rsub + 16 * p;
        c[p] = (row < rows) ? __ldg(reinterpret_cast<const uint2*>(codes + row * (K / 2) + col / 2)) : make_uint2(0, 0);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int rr = rsub + 16 * p;
        const int64_t row = row0 + rr;
        if (row >= rows) break;
        const uint32_t word = tile[128 * (blk >> 2) + scale_word_in_tile((uint32_t)rr)];
        const float gs = __fmul_rn(g, ue4m3_value((word >> (8 * (blk & 3))) & 0x7F));
        float v[16];
        uint32_t h[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            cvt_e2m1x8_to_f16x2(half ? c[p].y : c[p].x, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
                const float2 q = __fmul2_rn(f, make_float2(gs, gs));
                v[8 * half + 2 * e] = q.x;
                v[8 * half + 2 * e + 1] = q.y;
            }
        }
        if constexpr (F32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + row * K + col);
#pragma unroll
            for (int q = 0; q < 4; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + row * K + col);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// Column sums of bf16 rows [rows][cols] in fp32: CTA (x, y) sums 256 columns
// (8 per lane) of its share of the rows, its eight warps every eighth row;
// their sums meet in shared memory in warp order and the CTA writes one row of
// partial sums, which the second kernel adds in order.  No atomics, so the
// result does not depend on timing.
__global__ void __launch_bounds__(256) colsum_part_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld, int64_t rows,
                                                          int64_t cols, int64_t rows_per_cta, float* part) {
    __shared__ float sum[8][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 256 + 8 * lane;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_cta;
    const int64_t r1 = (r0 + rows_per_cta < rows) ? r0 + rows_per_cta : rows;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const bool whole = col + 8 <= cols;
    if (whole) {
#pragma unroll 4
        for (int64_t r = r0 + warp; r < r1; r += 8) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + r * ld + col));
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] += bf16lo(v[i]);
                acc[2 * i + 1] += bf16hi(v[i]);
            }
        }
    } else if (col < cols) {
        for (int64_t r = r0 + warp; r < r1; r += 8)
            for (int i = 0; i < 8; ++i)
                if (col + i < cols) acc[i] += __bfloat162float(x[r * ld + col + i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp][8 * lane + i] = acc[i];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c < cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sum[w][threadIdx.x];
        part[(int64_t)blockIdx.y * cols + c] = s;
    }
}

__global__ void __launch_bounds__(256) colsum_join_kernel(const float* __restrict__ part, int n, int64_t cols, float* out) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += part[(int64_t)i * cols + c];
    out[c] = s;
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantRowsArgs& a0, bool f32, cudaStream_t stream) {
    QuantRowsArgs a = a0;
    if (a.rows == 0) return cudaSuccess;
    a.n_part = 0;
    // up to this many values each CTA scans x itself: a second launch costs more
    if (a.dynamic && a.rows * a.K > 32768) {
        const int64_t want = (a.rows * a.K / 16 + 4 * QTHREADS - 1) / (4 * QTHREADS);
        a.n_part = (int)(want < ROWS_AMAX_PARTS ? want : ROWS_AMAX_PARTS);
        if (f32)
            rows_amax_kernel<true><<<a.n_part, QTHREADS, 0, stream>>>(a.x, a.ld, a.rows, a.K, a.part);
        else
            rows_amax_kernel<false><<<a.n_part, QTHREADS, 0, stream>>>(a.x, a.ld, a.rows, a.K, a.part);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((a.K + TILE_COLS - 1) / TILE_COLS), (unsigned)((a.rows + TILE_ROWS - 1) / TILE_ROWS));
    if (f32)
        quantize_rows_kernel<true><<<grid, QTHREADS, 0, stream>>>(a);
    else
        quantize_rows_kernel<false><<<grid, QTHREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_dequant_rows(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t rows, int64_t K,
                                void* out, bool f32, cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    const dim3 grid((unsigned)((K + TILE_COLS - 1) / TILE_COLS), (unsigned)((rows + TILE_ROWS - 1) / TILE_ROWS));
    if (f32)
        dequant_rows_kernel<true><<<grid, QTHREADS, 0, stream>>>(codes, scales, g, rows, K, out);
    else
        dequant_rows_kernel<false><<<grid, QTHREADS, 0, stream>>>(codes, scales, g, rows, K, out);
    return cudaGetLastError();
}

cudaError_t launch_column_sums(const __nv_bfloat16* x, int64_t ld, int64_t rows, int64_t cols, float* part, float* out,
                               cudaStream_t stream) {
    if (cols == 0) return cudaSuccess;
    if (rows == 0) return cudaMemsetAsync(out, 0, (size_t)cols * 4, stream);
    const int64_t strips = (cols + 255) / 256;
    int64_t n = (148 * 4 + strips - 1) / strips;  // about four CTAs per SM
    const int64_t most = (rows + 63) / 64;
    n = n < most ? n : most;
    n = n < COLSUM_PARTS ? n : COLSUM_PARTS;
    const int64_t per = (rows + n - 1) / n;
    n = (rows + per - 1) / per;
    colsum_part_kernel<<<dim3((unsigned)strips, (unsigned)n), 256, 0, stream>>>(x, ld, rows, cols, per, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    colsum_join_kernel<<<(unsigned)strips, 256, 0, stream>>>(part, (int)n, cols, out);
    return cudaGetLastError();
}

}  // namespace fp4attn
