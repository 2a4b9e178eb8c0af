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

constexpr int QTHREADS = 256;  // of the maxima and of reading back

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

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// Largest magnitude of a row segment per CTA.  The maxima go to a list, not to
// one word by atomics: the list needs no clearing before the call.
template <bool F32>
__global__ void __launch_bounds__(QTHREADS) rows_amax_kernel(const void* x, int64_t ld, int64_t rows, int64_t K,
                                                             float* part) {
    __shared__ float scratch[QTHREADS / 32];
    pdl_wait();
    pdl_trigger();
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

// The quantiser: one persistent CTA per SM goes through units of 128 rows x 128
// channels (two scale tiles), which bulk tensor copies bring into a ring of 192
// KB; a thread takes a block of 16 values of either tile.  The lanes of a warp
// stand for rows r, r + 1 of each 32-row quarter by the tile's four blocks:
// their eight scale words are one 32-byte sector, and the reads meet no bank
// conflicts.  8192 x 6144 bf16: 24 us (5.3 TB/s), two thirds of the issue slots.
constexpr int Q_CONSUMERS = 512;
constexpr int Q_THREADS = Q_CONSUMERS + 32;
template <bool F32>
struct QuantRing {
    static constexpr uint32_t BOX = 128 * 128;             // 128 rows of 128 bytes
    static constexpr uint32_t TILE = F32 ? 2 * BOX : BOX;  // 64 channels
    static constexpr uint32_t SLOT = 2 * TILE;
    static constexpr int SLOTS = F32 ? 3 : 6;
};
constexpr uint64_t kLimitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait
constexpr uint64_t kDrainNs = 200000000ull;

template <bool F32>
__global__ void __launch_bounds__(Q_THREADS, 1) quantize_rows_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                     const __grid_constant__ QuantRowsArgs a) {
    using R = QuantRing<F32>;
    constexpr int ES = F32 ? 4 : 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ ScaleTable table;
    __shared__ uint64_t full[R::SLOTS], empty[R::SLOTS];
    __shared__ float scratch[Q_CONSUMERS / 32];
    __shared__ int abort_all;
    // Behind the pass for the maxima, which has waited for whatever writes x, x
    // may be loaded at once: only the maxima themselves are waited for, by the
    // threads that read them.
    const bool behind_maxima = a.n_part > 0;
    if (!behind_maxima) {
        pdl_wait();
        pdl_trigger();
    }
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int chunks = (int)scale_chunks(a.K), units_wide = (chunks + 1) / 2;
    // units fit 31 bits (32768 row blocks by 8192); the last rows first: after a
    // pass for the maxima they are the ones still in L2
    const int units = (int)((a.rows + 127) / 128) * units_wide;
    const int first = units - 1 - (int)blockIdx.x, step = (int)gridDim.x;
    const int step_rb = step / units_wide, step_c = step - step_rb * units_wide;
    int rb = first / units_wide, c = first - rb * units_wide;  // row block and pair of chunks of this role's unit
    auto next_unit = [&]() {
        rb -= step_rb;
        c -= step_c;
        if (c < 0) {
            c += units_wide;
            --rb;
        }
    };
    volatile int* abort_flag = &abort_all;
    if (t == 0) {
        for (int s = 0; s < R::SLOTS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), Q_CONSUMERS / 32);
        }
        abort_all = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == Q_CONSUMERS / 32) {
        // ------------------------------------------------------ producer --
        if (lane == 0) {
            int it = 0;
            for (int u = first; u >= 0; u -= step, next_unit(), ++it) {
                const int slot = it % R::SLOTS;
                if (it >= R::SLOTS &&
                    !mbar_wait(smem_u32(&empty[slot]), (it / R::SLOTS - 1) & 1, abort_flag, a.status, kLimitNs))
                    break;
                const uint32_t bar = smem_u32(&full[slot]), at = smem_u32(ring) + R::SLOT * slot;
                const int tiles = 2 * c + 1 < chunks ? 2 : 1;
                mbar_arrive_expect_tx(bar, R::TILE * tiles);
                for (int i = 0; i < tiles * (int)(R::TILE / R::BOX); ++i)
                    tma_load_2d(at + R::BOX * i, &tm_x, 128 * c + 128 / ES * i, 128 * rb, bar);
            }
            if (*abort_flag)  // this CTA's own copies land before it leaves (bounded)
                for (int i = (it > R::SLOTS ? it - R::SLOTS : 0); i < it; ++i) {
                    int dummy = 0;
                    mbar_wait(smem_u32(&full[i % R::SLOTS]), (i / R::SLOTS) & 1, &dummy, nullptr, kDrainNs);
                }
        }
    } else {
        // ----------------------------------------------------- consumers --
        float g = 1.0f;
        if (a.dynamic) {
            // the maxima of the launch before, or (small inputs) all of x
            float m = 0.0f;
            if (behind_maxima) {
                pdl_wait();
                pdl_trigger();
                for (int i = t; i < a.n_part; i += Q_CONSUMERS) m = max_nan(m, __ldcg(a.part + i));
            } else {
                const int64_t per_row = a.K / 16;
                for (int64_t i = t; i < a.rows * per_row; i += Q_CONSUMERS) {
                    const int64_t r = i / per_row, b = i - r * per_row;
                    Block16<F32> x;
                    x.load(static_cast<const char*>(a.x) + (r * a.ld + b * 16) * ES);
                    float lo[8], hi[8];
                    x.values(lo, hi);
                    m = max_nan(m, amax16(lo, hi));
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) scratch[warp] = m;
            consumers_sync();
#pragma unroll
            for (int w = 0; w < Q_CONSUMERS / 32; ++w) m = max_nan(m, scratch[w]);
            g = computed_gscale(m);
            if (blockIdx.x == 0 && t == 0) *a.g_out = g;
        } else if (a.g) {
            g = __ldg(a.g);
        }
        if (blockIdx.x == 0 && t == 0 && bad_gscale(g)) raise_status(a.status, FP4ATTN_ERR_RANGE);
        make_scale_table(table, g, t);
        consumers_sync();
        const float guess = table.guess;
        const int blk = lane & 3, row_in = 2 * warp + ((lane >> 2) & 1) + 32 * (lane >> 3);
        const uint32_t sw = (uint32_t)row_in & 7u, word_in = scale_word_in_tile((uint32_t)row_in);
        const int rows_left = (int)(a.rows - row_in), half_k = (int)(a.K / 2);
        uint8_t* codes = a.codes + (int64_t)row_in * half_k + 8 * blk;
        uint32_t* words = reinterpret_cast<uint32_t*>(a.scales) + word_in;
        bool finite = true;
        int it = 0;
        for (int u = first; u >= 0; u -= step, next_unit(), ++it) {
            const int slot = it % R::SLOTS;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[slot]), (it / R::SLOTS) & 1, abort_flag, a.status, kLimitNs)))
                break;
            const int tiles = 2 * c + 1 < chunks ? 2 : 1;
            const uint8_t* at = ring + R::SLOT * slot + 128 * row_in;
            uint8_t* code_at = codes + ((int64_t)128 * rb * half_k + 64 * c);
            uint32_t* word_at = words + ((int64_t)rb * chunks + 2 * c) * 128;
            const bool row_on = 128 * rb < rows_left;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h >= tiles) break;
                const uint8_t* tile = at + R::TILE * h;
                float2 v[8];
                float m;
                if constexpr (F32) {
                    m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f =
                            *reinterpret_cast<const float4*>(tile + R::BOX * (blk >> 1) + 16u * ((4u * (blk & 1) + i) ^ sw));
                        v[2 * i] = make_float2(f.x, f.y);
                        v[2 * i + 1] = make_float2(f.z, f.w);
                        m = max_nan(m, max_nan(max_nan(fabsf(f.x), fabsf(f.y)), max_nan(fabsf(f.z), fabsf(f.w))));
                    }
                } else {
                    const uint4 lo = *reinterpret_cast<const uint4*>(tile + 16u * ((2u * blk) ^ sw));
                    const uint4 hi = *reinterpret_cast<const uint4*>(tile + 16u * ((2u * blk + 1) ^ sw));
                    const uint32_t m2 = max_pair(amax_pair(lo), amax_pair(hi));
                    m = max_nan(bf16lo(m2), bf16hi(m2));
                    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = make_float2(bf16lo(w[i]), bf16hi(w[i]));
                }
                if (h == tiles - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));  // the warp's values are in registers
                }
                finite = finite && (m < INFINITY);
                uint32_t s;
                float inv;
                row_block_scale(table, guess, m, g, s, inv);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(v[i], make_float2(inv, inv));
                const uint32_t c0 = cvt_e2m1x8(v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y);
                const uint32_t c1 = cvt_e2m1x8(v[4].x, v[4].y, v[5].x, v[5].y, v[6].x, v[6].y, v[7].x, v[7].y);
                if (row_on && 64 * (2 * c + h) + 16 * blk < 2 * half_k &&
                    FP4ATTN_IN_BOUNDS(code_at + 32 * h + 8 <= a.codes + a.rows * half_k, a.status))
                    *reinterpret_cast<uint2*>(code_at + 32 * h) = make_uint2(c0, c1);
                // four blocks of a row make a word of the tile
                uint32_t word = s << (8 * blk);
                word |= __shfl_xor_sync(0xffffffffu, word, 1);
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
                if (blk == 0 && FP4ATTN_IN_BOUNDS(u < units, a.status)) word_at[128 * h] = word;
            }
        }
        if (!finite) raise_status(a.status, FP4ATTN_ERR_RANGE);
    }
}

// The values of quantised rows: fl(fl(g s) * e2m1), to fp32 or rounded to bf16
// (exact in bf16 for g a power of two).  A CTA reads back 128 rows x 128
// channels, a thread eight values (16 bytes of bf16, so that a warp's store
// fills whole sectors) of every sixteenth row.  8192 x 6144: 20 us, 6.4 TB/s (32
// us with 32 bytes a thread, half a sector an instruction).
template <bool F32>
__device__ __forceinline__ void dequant_tile(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                             const float* gp, int64_t rows, int64_t K, void* out, int64_t rb, int64_t cb) {
    const int t = threadIdx.x;
    const int64_t chunks = scale_chunks(K);
    const int64_t col = cb * 128 + 8 * (t & 15);
    if (col >= K) return;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(scales) + (rb * chunks + col / 64) * 128;
    const int row_in = t >> 4, shift = 8 * ((t >> 1) & 3);
    const int n = (int)(rows - 128 * rb < 128 ? rows - 128 * rb : 128);  // rows of this block
    const uint8_t* src = codes + (128 * rb + row_in) * (K / 2) + col / 2;
    uint32_t c[8], w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = row_in + 16 * p;
        c[p] = w[p] = 0;
        if (r < n) {
            c[p] = __ldg(reinterpret_cast<const uint32_t*>(src + (int64_t)16 * p * (K / 2)));
            w[p] = __ldg(words + scale_word_in_tile((uint32_t)r));
        }
    }
    const float g = gp ? __ldg(gp) : 1.0f;
    char* dst = static_cast<char*>(out) + ((128 * rb + row_in) * K + col) * (F32 ? 4 : 2);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        if (row_in + 16 * p < n) {
            const float gs = __fmul_rn(g, ue4m3_value((w[p] >> shift) & 0x7F));
            uint32_t h[4];
            cvt_e2m1x8_to_f16x2(c[p], h);
            float2 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h[e])), make_float2(gs, gs));
            char* at = dst + (int64_t)16 * p * K * (F32 ? 4 : 2);
            if constexpr (F32) {
                reinterpret_cast<float4*>(at)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
                reinterpret_cast<float4*>(at)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
            } else {
                *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                           pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
            }
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(QTHREADS) dequant_rows_kernel(const uint8_t* codes, const uint8_t* scales, const float* gp,
                                                                int64_t rows, int64_t K, void* out) {
    pdl_wait();
    pdl_trigger();
    dequant_tile<F32>(codes, scales, gp, rows, K, out, blockIdx.y, blockIdx.x);
}

// Column sums of bf16 rows [rows][cols] in fp32, strip `strip` of 256 columns (8
// per lane) and rows [r0, r1): the warps take every eighth row, their sums meet
// in shared memory in warp order and leave as one row of partial sums, which are
// added in order later.  No atomics, so the result does not depend on timing.
__device__ __forceinline__ void colsum_part(const __nv_bfloat16* __restrict__ x, int64_t ld, int64_t cols, int64_t strip,
                                            int64_t r0, int64_t r1, float* part, float (&sum)[8][256]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = strip * 256 + 8 * lane;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (col + 8 <= cols) {
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
    const int64_t c = strip * 256 + threadIdx.x;
    if (c < cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sum[w][threadIdx.x];
        part[c] = s;
    }
}

// What the linear layer's backward needs before its products, in one launch:
// the unit-scale values of w and x, and the partial column sums of dy.
__global__ void __launch_bounds__(QTHREADS) backward_prepare_kernel(const __grid_constant__ LinearBwdArgs a,
                                                                    const __grid_constant__ BwdPrepare n) {
    __shared__ float sum[8][256];
    pdl_wait();
    pdl_trigger();
    int b = blockIdx.x;
    if (b < n.sums) {  // first: they read the most
        const int part = b / n.strips, strip = b - part * n.strips;
        const int64_t r0 = n.rows_per_part * part, r1 = r0 + n.rows_per_part;
        colsum_part(a.dy, a.ld_dy, a.N, strip, r0, r1 < a.M ? r1 : a.M, a.colsum_part + (int64_t)part * a.N, sum);
        return;
    }
    b -= n.sums;
    const int wide = (int)((a.K + 127) / 128);
    const bool is_w = b < n.w_tiles;
    if (!is_w) b -= n.w_tiles;
    const int rb = b / wide, cb = b - rb * wide;
    dequant_tile<false>(is_w ? a.w_codes : a.x_codes, is_w ? a.w_scales : a.x_scales, nullptr, is_w ? a.N : a.M, a.K,
                        is_w ? a.w_bf16 : a.x_bf16, rb, cb);
}

}  // namespace

namespace {

template <bool F32>
cudaError_t launch_quantize(const QuantRowsArgs& a, cudaStream_t stream) {
    using R = QuantRing<F32>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // rows x 128 bytes, what lies past the matrix's ends reads as zero
    CUtensorMap tm;
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.rows};
    const uint64_t strides[1] = {(uint64_t)a.ld * (F32 ? 4 : 2)};
    const uint32_t box[2] = {F32 ? 32u : 64u, 128};
    if (!encode_tensor_map(&tm, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                           const_cast<void*>(a.x), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    constexpr size_t smem = (size_t)R::SLOT * R::SLOTS + 1024;
    auto kernel = quantize_rows_kernel<F32>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (a.rows + 127) / 128 * ((scale_chunks(a.K) + 1) / 2);
    return launch_behind(kernel, dim3((unsigned)(units < sms ? units : sms)), Q_THREADS, smem, stream, 1, tm, a);
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
        const cudaError_t e = launch_behind(f32 ? rows_amax_kernel<true> : rows_amax_kernel<false>, dim3(a.n_part), QTHREADS, 0,
                                            stream, 1, a.x, a.ld, a.rows, a.K, a.part);
        if (e != cudaSuccess) return e;
    }
    return f32 ? launch_quantize<true>(a, stream) : launch_quantize<false>(a, stream);
}

cudaError_t launch_dequant_rows(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t rows, int64_t K,
                                void* out, bool f32, cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    const dim3 grid((unsigned)((K + 127) / 128), (unsigned)((rows + 127) / 128));
    return launch_behind(f32 ? dequant_rows_kernel<true> : dequant_rows_kernel<false>, grid, QTHREADS, 0, stream, 1, codes,
                         scales, g, rows, K, out);
}

cudaError_t launch_backward_prepare(const LinearBwdArgs& a, int& colsum_parts, cudaStream_t stream) {
    BwdPrepare n{};
    const int64_t wide = (a.K + 127) / 128;
    n.w_tiles = a.dx ? (int)((a.N + 127) / 128 * wide) : 0;
    const int64_t x_tiles = a.dw ? (a.M + 127) / 128 * wide : 0;
    colsum_parts = 0;
    if (a.dbias) {
        n.strips = (int)((a.N + 255) / 256);
        int64_t parts = (148 * 4 + n.strips - 1) / n.strips;  // about four CTAs per SM
        const int64_t most = (a.M + 63) / 64;
        parts = parts < most ? parts : most;
        parts = parts < COLSUM_PARTS ? parts : COLSUM_PARTS;
        n.rows_per_part = (a.M + parts - 1) / parts;
        colsum_parts = (int)((a.M + n.rows_per_part - 1) / n.rows_per_part);
        n.sums = n.strips * colsum_parts;
    }
    return launch_behind(backward_prepare_kernel, dim3((unsigned)(n.sums + n.w_tiles + x_tiles)), QTHREADS, 0, stream, 1, a, n);
}

}  // namespace fp4attn
