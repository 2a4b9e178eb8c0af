// The NVFP4 product of the linear layers: out[m][n] = g_x g_w sum_k x[m][k] w[n][k] + bias[n].
//
// FastVideo "Pika H3 Flex in FastVideo", section "NVFP4 QAD": every attention
// and feed-forward linear takes 4-bit weights and activations with an 8-bit
// scale per 16 values.  One persistent kernel on the block-scaled FP4 tensor
// cores:
//   * a tile is 128 rows of one operand (the lanes of TMEM) by TN rows of the
//     other (its columns).  Small products run on single CTAs with the weight on
//     the lanes: a warp then stores 32 consecutive outputs, and rows of y may
//     start anywhere.  Large ones run on pairs of CTAs (below);
//   * K goes by in stages of 256 values (128 code bytes: 128B-swizzled K-major
//     tiles by TMA, and whole scale tiles by bulk copies) through a ring;
//   * per stage the MMA warp copies the scale tiles to TMEM and issues one
//     M=128, N=TN, K=64 tcgen05.mma for each 64 values;
//   * two accumulators alternate, so the epilogue of one tile runs under the
//     products of the next;
//   * SPLIT: few tiles and a long K.  A cluster shares one tile, each CTA a
//     part of K; the fp32 parts are added in rank order through distributed
//     shared memory, so the result does not depend on timing.
// Every wait is bounded; a wait that runs out raises FP4ATTN_ERR_TIMEOUT in the
// status word and the CTA winds down.
#include <cuda_bf16.h>

#include "fp4_operands.cuh"
#include "nvfp4_rows.cuh"
#include "tile_store.cuh"

namespace fp4attn {

namespace {

constexpr int BP = 128;       // rows of the lane-side operand per tile
constexpr int BK = 256;       // K per stage
constexpr int CHUNKS = BK / 64;
constexpr int THREADS = 192;  // warps 0-3 epilogue, 4 producer, 5 MMA
constexpr int WARP_PRODUCER = 4, WARP_MMA = 5;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL = 448;  // scale factors: per 64-chunk 4 columns of the lane side, 4 or 8 of the other
constexpr uint64_t kLimitNs = 2000000000ull;   // 2 s: far beyond any legitimate wait
constexpr uint64_t kDrainNs = 200000000ull;    // 0.2 s for the wind-down waits

__host__ __device__ constexpr int round128(int n) { return (n + 127) / 128 * 128; }

template <int TN>
struct Cfg {
    static constexpr uint32_t P_BYTES = BP * BK / 2;
    static constexpr uint32_t Q_BYTES = (uint32_t)(TN * BK / 2 + 1023) / 1024 * 1024;
    static constexpr uint32_t SFP_BYTES = CHUNKS * 512;
    static constexpr uint32_t SFQ_BYTES = (uint32_t)(round128(TN) / 128) * CHUNKS * 512;
    static constexpr uint32_t STAGE = P_BYTES + Q_BYTES + SFP_BYTES + SFQ_BYTES;
    static constexpr int STAGES = (int)((222u * 1024) / STAGE) < 8 ? (int)((222u * 1024) / STAGE) : 8;
    static constexpr uint32_t ACC1 = TN;  // first column of the second accumulator
    static constexpr int SFQ_COLS = round128(TN) / 32;
    static_assert(ACC1 + TN <= SF_COL, "TMEM: accumulators end before the scale factors");
    static_assert(SF_COL + CHUNKS * (4 + SFQ_COLS) <= TMEM_COLS, "TMEM: scale factors");
    static_assert(STAGE % 1024 == 0, "stages keep the swizzle's alignment");
};

struct Bars {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2];
    uint64_t next_ok;
    uint64_t final_;
    uint32_t tmem_base;
    int abort_flag;
};

struct GemmParams {
    int P, Q;              // rows of the lane-side and of the column-side operand
    int p_tiles, q_tiles;
    int stages;            // K in stages of 256
    int chunks;            // K in chunks of 64
    const uint8_t* sfp;
    const uint8_t* sfq;
    int sfp_blocks, sfq_blocks;  // 128-row blocks of the two scale arrays
    const float* gx;
    const float* gw;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    long long ld;
    int N;
    int weight_ready;  // the weight may be loaded before the kernel in front has finished
    int* status;
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, kLimitNs));
}
__device__ __forceinline__ bool drain_wait(uint32_t bar, uint32_t parity) {
    int dummy = 0;
    return mbar_wait(bar, parity, &dummy, nullptr, kDrainNs);
}

// Tiles in groups of 8 lane-side tiles, the group's column tiles outermost: a
// wave of 148 tiles then reads about 8 + 18 operand tiles, not 148 of one side.
constexpr int GROUP = 8;
__device__ __forceinline__ void tile_of(int t, int p_tiles, int q_tiles, int& pt, int& qt) {
    const int per = GROUP * q_tiles;
    const int grp = t / per, in = t - grp * per;
    const int rows = min(GROUP, p_tiles - grp * GROUP);
    qt = in / rows;
    pt = grp * GROUP + (in - qt * rows);
}

__device__ __forceinline__ uint64_t rows_desc(uint32_t addr) { return smem_desc(addr, 16, 1024, LAYOUT_SW128); }

// g_x g_w as g * pre.  Either scale may be any positive number; where their product
// leaves fp32's normal range, pre is a power of two that brings g back into it.  A
// sum of products is 0 or lies between 2^-20 and 2^43, so that sum * pre is exact
// for |log2 pre| <= 64, and past that every nonzero result is outside bf16's range
// (a zero one stays zero: g is finite).
struct OutScale {
    float g, pre;
};
__device__ __forceinline__ OutScale out_scale(float gx, float gw) {
    const float g = __fmul_rn(gx, gw);
    if (g >= 1.17549435e-38f && g <= 3.40282347e38f) return {g, 1.0f};
    const double both = (double)gx * (double)gw;  // exact
    const int e = ilogb(both);                    // of a bad scale anything: it is reported
    const int k = e < -126 ? max(e + 126, -64) : e > 126 ? min(e - 126, 64) : 0;
    return {fminf((float)ldexp(both, -k), 3.40282347e38f), ldexpf(1.0f, k)};
}
template <int W>
__device__ __forceinline__ void prescale(uint32_t (&r)[W], float pre) {
    if (pre != 1.0f)
#pragma unroll
        for (int k = 0; k < W; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * pre);
}

// Lane = column n of the output, W of its rows from m0 in one thread.
template <int W>
__device__ __forceinline__ void store_columns(const GemmParams& p, const uint32_t (&r)[W], float g, float bias, int n,
                                              int m0) {
    if (n >= p.P) return;
    __nv_bfloat16* dst = p.out + (long long)m0 * p.ld + n;
    const long long ld = p.ld;
    if (m0 + W <= p.Q && FP4ATTN_IN_BOUNDS(n < p.N, p.status)) {
#pragma unroll
        for (int k = 0; k < W; ++k, dst += ld) *dst = __float2bfloat16_rn(__fmaf_rn(__uint_as_float(r[k]), g, bias));
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k, dst += ld)
            if (m0 + k < p.Q && FP4ATTN_IN_BOUNDS(n < p.N, p.status))
                *dst = __float2bfloat16_rn(__fmaf_rn(__uint_as_float(r[k]), g, bias));
    }
}

template <int TN, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                    const GemmParams p) {
    using C = Cfg<TN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars sm;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_u = smem_u32(ring);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = p.p_tiles * p.q_tiles;
    // SPLIT: the CTAs of a cluster share tile blockIdx.x / S
    uint32_t rank = 0, ranks = 1;
    if constexpr (SPLIT) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    }
    const int first = SPLIT ? (int)(blockIdx.x / ranks) : (int)blockIdx.x;
    const int step = SPLIT ? n_tiles : (int)gridDim.x;
    const int s_begin = SPLIT ? (int)((long long)p.stages * rank / ranks) : 0;
    const int s_end = SPLIT ? (int)((long long)p.stages * (rank + 1) / ranks) : p.stages;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        mbar_init(smem_u32(&sm.acc_full[0]), 1);
        mbar_init(smem_u32(&sm.acc_full[1]), 1);
        mbar_init(smem_u32(&sm.next_ok), 4);
        mbar_init(smem_u32(&sm.final_), 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == WARP_PRODUCER && lane == 0) {
        prefetch_tmap(&tm_p);
        prefetch_tmap(&tm_q);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort_flag = &sm.abort_flag;

    if (warp == WARP_PRODUCER) {
        // ------------------------------------------------------ producer --
        // x may still be written by the launch in front: where the weight is not
        // (the linear layer's own quantiser), its first stages go out before that
        // launch is waited for.
        int it = 0;
        bool waited = p.weight_ready == 0;
        if (waited) pdl_wait();
        auto copy_p = [&](int slot, int ks, int pt) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            const uint32_t at = ring_u + C::STAGE * slot;
            const int n = min(CHUNKS, p.chunks - CHUNKS * ks);
            tma_load_2d(at, &tm_p, 128 * ks, BP * pt, full);
            bulk_load(at + C::P_BYTES + C::Q_BYTES, p.sfp + ((long long)pt * p.chunks + CHUNKS * ks) * 512, 512u * n,
                      full);
        };
        auto copy_q = [&](int slot, int ks, int qt) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            const uint32_t at = ring_u + C::STAGE * slot;
            const int n = min(CHUNKS, p.chunks - CHUNKS * ks);
            tma_load_2d(at + C::P_BYTES, &tm_q, 128 * ks, TN * qt, full);
#pragma unroll
            for (int b = 0; b < round128(TN) / 128; ++b) {
                const int rb = qt * (round128(TN) / 128) + b;
                if (rb < p.sfq_blocks)
                    bulk_load(at + C::P_BYTES + C::Q_BYTES + C::SFP_BYTES + CHUNKS * 512 * b,
                              p.sfq + ((long long)rb * p.chunks + CHUNKS * ks) * 512, 512u * n, full);
            }
        };
        auto bytes_of = [&](int ks, int qt) {
            const int n = min(CHUNKS, p.chunks - CHUNKS * ks);
            const int blocks = min(round128(TN) / 128, p.sfq_blocks - qt * (round128(TN) / 128));
            return C::P_BYTES + (uint32_t)(TN * BK / 2) + 512u * n * (1 + blocks);
        };
        bool ok = true;
        for (int t = first; ok && t < n_tiles; t += step) {
            int pt, qt;
            tile_of(t, p.p_tiles, p.q_tiles, pt, qt);
            int ks = s_begin;
            if (!waited) {
                // the ring is empty: fill it with weight copies, wait, then x's
                const int pre = min(C::STAGES, s_end - s_begin);
                if (lane == 0) {
                    for (int i = 0; i < pre; ++i) {
                        mbar_arrive_expect_tx(smem_u32(&sm.full[i]), bytes_of(ks + i, qt));
                        copy_p(i, ks + i, pt);
                    }
                }
                pdl_wait();
                if (lane == 0) {
                    for (int i = 0; i < pre; ++i) copy_q(i, ks + i, qt);
                }
                __syncwarp();
                waited = true;
                it = pre;
                ks += pre;
            }
            for (; ks < s_end; ++ks, ++it) {
                const int slot = it % C::STAGES;
                if (it >= C::STAGES &&
                    !warp_wait(smem_u32(&sm.empty[slot]), (it / C::STAGES - 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_u32(&sm.full[slot]), bytes_of(ks, qt));
                    copy_p(slot, ks, pt);
                    copy_q(slot, ks, qt);
                }
                __syncwarp();
            }
        }
        if (!waited) pdl_wait();
        if (lane == 0 && *abort_flag) {
            // wind down: this CTA's own copies land before it exits
            for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it; ++i)
                drain_wait(smem_u32(&sm.full[i % C::STAGES]), (i / C::STAGES) & 1);
        }
    } else if (warp == WARP_MMA) {
        // ----------------------------------------------------------- MMA --
        const bool leader = elect_one_sync();
        constexpr uint32_t IDESC = idesc_mxf4(BP, TN);
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, p.status, kLimitNs));
        };
        int it = 0, local = 0;
        bool ok = true;
        for (int t = first; ok && t < n_tiles; t += step, ++local) {
            const uint32_t acc = tmem + (local & 1 ? C::ACC1 : 0u);
            // the tile before has left the columns this one starts on (and
            // with it every earlier tile all of its own)
            if (local > 0 && !wait(smem_u32(&sm.next_ok), (local - 1) & 1)) break;
            tc_fence_after();
            for (int ks = s_begin; ks < s_end; ++ks, ++it) {
                const int slot = it % C::STAGES;
                if (!wait(smem_u32(&sm.full[slot]), (it / C::STAGES) & 1)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    tc_fence_after();
                    const uint32_t at = ring_u + C::STAGE * slot;
                    const uint32_t sf = at + C::P_BYTES + C::Q_BYTES;
                    const int n = min(CHUNKS, p.chunks - CHUNKS * ks);
                    const uint64_t pd = rows_desc(at), qd = rows_desc(at + C::P_BYTES);
#pragma unroll
                    for (int c = 0; c < CHUNKS; ++c) {
                        if (c < n) {
                            // one thread's copies and products run in the order issued
                            const uint32_t ta = tmem + SF_COL + 4u * c;
                            const uint32_t tb = tmem + SF_COL + 4u * CHUNKS + (uint32_t)C::SFQ_COLS * c;
                            tmem_cp_32x128b_x4(ta, smem_desc(sf + 512 * c, 0, 128, LAYOUT_NONE));
#pragma unroll
                            for (int b = 0; b < round128(TN) / 128; ++b)
                                tmem_cp_32x128b_x4(tb + 4u * b, smem_desc(sf + C::SFP_BYTES + CHUNKS * 512 * b + 512 * c,
                                                                          0, 128, LAYOUT_NONE));
                            mma_mxf4nvf4(acc, pd + 2u * c, qd + 2u * c, IDESC, ta, tb, (ks > s_begin || c > 0) ? 1u : 0u);
                        }
                    }
                    tc_commit(smem_u32(&sm.empty[slot]));
                    if (ks == s_end - 1) tc_commit(smem_u32(&sm.acc_full[local & 1]));
                }
                __syncwarp();
            }
        }
        // every product this warp issued must finish before TMEM is freed
        if (leader) {
            tc_commit(smem_u32(&sm.final_));
            drain_wait(smem_u32(&sm.final_), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue --
        pdl_wait();
        pdl_trigger();
        const float gx = p.gx ? __ldcg(p.gx) : 1.0f, gw = p.gw ? __ldg(p.gw) : 1.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (bad_gscale(gx) || bad_gscale(gw)))
            raise_status(p.status, FP4ATTN_ERR_RANGE);
        const OutScale g = out_scale(gx, gw);
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const int row = 32 * warp + lane;
        int local = 0;
        for (int t = first; t < n_tiles; t += step, ++local) {
            int pt, qt;
            tile_of(t, p.p_tiles, p.q_tiles, pt, qt);
            const uint32_t acc = tmem + lanes + (local & 1 ? C::ACC1 : 0u);
            if (!warp_wait(smem_u32(&sm.acc_full[local & 1]), (local >> 1) & 1, abort_flag, p.status)) break;
            tc_fence_after();
            const int pr = BP * pt + row;  // this thread's row of the lane side
            const int q0 = TN * qt;
            if constexpr (SPLIT) {
                // the ring is idle now (every product of this CTA is done): the
                // part goes there column by column, 128 rows each
                float* part = reinterpret_cast<float*>(ring);
#pragma unroll 1
                for (int c0 = 0; c0 < TN; c0 += 16) {
                    uint32_t r[16];
                    tmem_ld16(acc + c0, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c0 + i) * BP + row] = __uint_as_float(r[i]);
                }
            } else {
                constexpr int W = TN < 32 ? 16 : 32;  // columns per step
                // the accumulators do not overlap: being here shows that this warp is
                // done with the tile before, which is all that the next one waits for
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.next_ok));
                const float own_bias = (p.bias && pr < p.P) ? __bfloat162float(p.bias[pr]) : 0.0f;
#pragma unroll 1
                for (int c0 = 0; c0 < TN; c0 += W) {
                    uint32_t r[W];
                    if constexpr (W == 16) tmem_ld16(acc + c0, r); else tmem_ld32(acc + c0, r);
                    tmem_wait_ld();
                    prescale(r, g.pre);
                    store_columns<W>(p, r, g.g, own_bias, pr, q0 + c0);
                    __syncwarp();
                }
            }
        }
        if constexpr (SPLIT) tc_fence_before();
    }

    if constexpr (SPLIT) {
        // Every CTA's part is in its shared memory; rank r adds columns
        // [r TN / ranks, (r + 1) TN / ranks) over the ranks in order.
        __syncwarp();
        cluster_sync();
        if (warp < 4) {
            const float gx = p.gx ? __ldcg(p.gx) : 1.0f, gw = p.gw ? __ldg(p.gw) : 1.0f;
            const OutScale g = out_scale(gx, gw);
            int pt, qt;
            tile_of(first, p.p_tiles, p.q_tiles, pt, qt);
            const int row = threadIdx.x;  // 0..127
            const int pr = BP * pt + row;
            const float bias = (p.bias && pr < p.P) ? __bfloat162float(p.bias[pr]) : 0.0f;
            const uint32_t part = ring_u + 4u * row;
            const int c_end = (int)(TN * (rank + 1) / ranks);
            // columns in eights: their loads from another CTA are on their way together
            for (int c = (int)(TN * rank / ranks); c < c_end; c += 8) {
                if (TN * qt + c >= p.Q) break;
                float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (uint32_t k = 0; k < ranks; ++k) {
                    const uint32_t at = mapa(part, k);
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = ld_cluster(at + 4u * BP * min(c + i, TN - 1));
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] += v[i];
                }
                if (pr < p.P)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int m = TN * qt + c + i;
                        if (c + i < c_end && m < p.Q &&
                            FP4ATTN_IN_BOUNDS((long long)m * p.ld + pr <= (long long)(p.Q - 1) * p.ld + p.N - 1, p.status))
                            p.out[(long long)m * p.ld + pr] = __float2bfloat16_rn(__fmaf_rn(s[i] * g.pre, g.g, bias));
                    }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its part
    }
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------ CTA pairs --
//
// Large products: a pair of CTAs owns a 256 x 256 tile (tcgen05 cta_group::2).
// Each CTA loads 128 rows of the lane side and 128 of the column side per stage
// and both read each other's half of the latter through the pair: 8 KB of codes
// in and 8 KB read per 128 clocks of tensor work, where a single CTA's 128 x 256
// tile needs 12 and 12.  The scales of the column side are wanted whole by both.
// The CTA of rank 0 issues the products; accumulators and scale factors lie in
// TMEM as in the kernel above.
//
// 109568 x 6144 x 6144: 1.58 ms, 5.2 PFLOP/s (1.85 ms on single CTAs).  A stage's
// products take 512 clocks and its 38 KB come from L2 in about 900 (42 bytes a
// clock and SM, 12 TB/s in all): on operands at rest the same loop reaches 7.4
// PFLOP/s at K = 24576.  Larger tiles do not fit TMEM beside the scale factors.

constexpr int PAIR_TILE = 256;
constexpr int PAIR_THREADS = 32 * (STORE_WARPS + 2);
constexpr int PAIR_PRODUCER = STORE_WARPS, PAIR_MMA = STORE_WARPS + 1;
struct PairCfg {
    static constexpr uint32_t P_BYTES = 128 * BK / 2;
    static constexpr uint32_t SFP_BYTES = CHUNKS * 512, SFQ_BYTES = 2 * CHUNKS * 512;
    static constexpr uint32_t STAGE = 2 * P_BYTES + SFP_BYTES + SFQ_BYTES;
    static constexpr int STAGES = 5;
    static constexpr uint32_t ACC1 = 192;  // the second accumulator shares 64 columns with the first
    static_assert(STAGE % 1024 == 0, "stages keep the swizzle's alignment");
    static_assert(SF_COL + CHUNKS * 12 <= TMEM_COLS, "TMEM: scale factors");
};

template <bool SWAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_sfp, const __grid_constant__ CUtensorMap tm_sfq,
                         const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ GemmParams p) {
    using C = PairCfg;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars sm;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_u = smem_u32(ring);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int n_tiles = p.p_tiles * p.q_tiles;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        mbar_init(smem_u32(&sm.acc_full[0]), 1);
        mbar_init(smem_u32(&sm.acc_full[1]), 1);
        mbar_init(smem_u32(&sm.next_ok), 2 * STORE_WARPS);  // the epilogue warps of both CTAs
        mbar_init(smem_u32(&sm.final_), 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == PAIR_MMA) {
        tmem_alloc_2cta(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish_2cta();
    }
    if (warp == PAIR_PRODUCER && lane == 0) {
        prefetch_tmap(&tm_p);
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_sfp);
        prefetch_tmap(&tm_sfq);
        if (!SWAP) prefetch_tmap(&tm_out);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort_flag = &sm.abort_flag;
    pdl_wait();
    pdl_trigger();

    if (warp == PAIR_PRODUCER) {
        // ------------------------------------------------------ producer --
        int it = 0;
        bool ok = true;
        for (int t = first; ok && t < n_tiles; t += step) {
            int pt, qt;
            tile_of(t, p.p_tiles, p.q_tiles, pt, qt);
            for (int ks = 0; ks < p.stages; ++ks, ++it) {
                const int slot = it % C::STAGES;
                if (it >= C::STAGES &&
                    !warp_wait(smem_u32(&sm.empty[slot]), (it / C::STAGES - 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    // the pair's copies all count on the first CTA's barrier; what lies
                    // past an operand's end comes as zeros and counts too
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[slot]), 2 * C::STAGE);
                    const uint32_t full = mapa(smem_u32(&sm.full[slot]), 0);
                    const uint32_t at = ring_u + C::STAGE * slot;
                    tma_load_2d_2cta(at, &tm_p, 128 * ks, PAIR_TILE * pt + 128 * rank, full);
                    tma_load_2d_2cta(at + C::P_BYTES, &tm_q, 128 * ks, PAIR_TILE * qt + 128 * rank, full);
                    tma_load_3d_2cta(at + 2 * C::P_BYTES, &tm_sfp, 0, CHUNKS * ks, 2 * pt + rank, full);
                    tma_load_3d_2cta(at + 2 * C::P_BYTES + C::SFP_BYTES, &tm_sfq, 0, CHUNKS * ks, 2 * qt, full);
                }
                __syncwarp();
            }
        }
        if (rank == 0 && lane == 0 && *abort_flag)
            for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it; ++i)
                drain_wait(smem_u32(&sm.full[i % C::STAGES]), (i / C::STAGES) & 1);
    } else if (warp == PAIR_MMA) {
        // ----------------------------------------------------------- MMA --
        if (rank == 0) {
            const bool leader = elect_one_sync();
            constexpr uint32_t IDESC = idesc_mxf4(PAIR_TILE, PAIR_TILE);
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, p.status, kLimitNs));
            };
            int it = 0, local = 0;
            bool ok = true;
            for (int t = first; ok && t < n_tiles; t += step, ++local) {
                const uint32_t acc = tmem + (local & 1 ? C::ACC1 : 0u);
                if (local > 0 && !wait(smem_u32(&sm.next_ok), (local - 1) & 1)) break;
                tc_fence_after();
                for (int ks = 0; ks < p.stages; ++ks, ++it) {
                    const int slot = it % C::STAGES;
                    if (!wait(smem_u32(&sm.full[slot]), (it / C::STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        tc_fence_after();
                        const uint32_t at = ring_u + C::STAGE * slot;
                        const uint32_t sf = at + 2 * C::P_BYTES;
                        const int n = min(CHUNKS, p.chunks - CHUNKS * ks);
                        const uint64_t pd = rows_desc(at), qd = rows_desc(at + C::P_BYTES);
#pragma unroll
                        for (int c = 0; c < CHUNKS; ++c) {
                            if (c < n) {
                                const uint32_t ta = tmem + SF_COL + 4u * c, tb = tmem + SF_COL + 4u * CHUNKS + 8u * c;
                                tmem_cp_32x128b_x4_2cta(ta, smem_desc(sf + 512 * c, 0, 128, LAYOUT_NONE));
#pragma unroll
                                for (int b = 0; b < 2; ++b)
                                    tmem_cp_32x128b_x4_2cta(
                                        tb + 4u * b,
                                        smem_desc(sf + C::SFP_BYTES + CHUNKS * 512 * b + 512 * c, 0, 128, LAYOUT_NONE));
                                mma_mxf4nvf4_2cta(acc, pd + 2u * c, qd + 2u * c, IDESC, ta, tb, (ks > 0 || c > 0) ? 1u : 0u);
                            }
                        }
                        tc_commit_2cta(smem_u32(&sm.empty[slot]));
                        if (ks == p.stages - 1) tc_commit_2cta(smem_u32(&sm.acc_full[local & 1]));
                    }
                    __syncwarp();
                }
            }
            if (leader) {
                tc_commit_2cta(smem_u32(&sm.final_));
                drain_wait(smem_u32(&sm.final_), 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------ epilogue --
        const float gx = p.gx ? __ldcg(p.gx) : 1.0f, gw = p.gw ? __ldg(p.gw) : 1.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (bad_gscale(gx) || bad_gscale(gw)))
            raise_status(p.status, FP4ATTN_ERR_RANGE);
        const OutScale scale = out_scale(gx, gw);
        const float g = scale.g;
        // a warp reads its quarter of the lanes and half of the columns, 64 at a time
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t box = ring_u + C::STAGES * C::STAGE + STORE_BOX * warp;
        int local = 0;
        for (int t = first; t < n_tiles; t += step, ++local) {
            int pt, qt;
            tile_of(t, p.p_tiles, p.q_tiles, pt, qt);
            const uint32_t acc = tmem + lanes + (local & 1 ? C::ACC1 : 0u);
            if (!warp_wait(smem_u32(&sm.acc_full[local & 1]), (local >> 1) & 1, abort_flag, p.status)) break;
            tc_fence_after();
            const int p0 = PAIR_TILE * pt + 128 * rank + 32 * quarter, pr = p0 + lane;
            const float own_bias = (SWAP && p.bias && pr < p.P) ? __bfloat162float(p.bias[pr]) : 0.0f;
            // The next tile's products wait for the columns that the accumulators
            // share (the last 64 of the first, the first 64 of the second), and for
            // every column of the tile before: each warp reports when it has read
            // what it has of the former, which shows that it is done with the latter.
            const bool last_first = !(local & 1) && half == 1;  // its second 64 columns are shared
            const bool shares = last_first || ((local & 1) && half == 0);
            auto report = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&sm.next_ok), 0));
            };
            if (!shares) report();
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int c0 = 128 * half + 64 * (i ^ (int)last_first), q0 = PAIR_TILE * qt + c0;
                uint32_t r[2][32];
                tmem_ld32(acc + c0, r[0]);
                tmem_ld32(acc + c0 + 32, r[1]);
                tmem_wait_ld();
                if (i == 0 && shares) report();
                prescale(r[0], scale.pre);
                prescale(r[1], scale.pre);
                if constexpr (SWAP) {
                    store_columns<32>(p, r[0], g, own_bias, pr, q0);
                    store_columns<32>(p, r[1], g, own_bias, pr, q0 + 32);
                } else {
                    uint32_t w[32];
                    if (p.bias) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            // N is even here: a pair of biases is there whole or not at all
                            const uint32_t b =
                                q0 + 2 * k < p.Q ? __ldg(reinterpret_cast<const uint32_t*>(p.bias + q0) + k) : 0u;
                            w[k] = pack_bf16x2(__fmaf_rn(__uint_as_float(r[k / 16][2 * (k % 16)]), g, bf16lo(b)),
                                               __fmaf_rn(__uint_as_float(r[k / 16][2 * (k % 16) + 1]), g, bf16hi(b)));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(r[k / 16][2 * (k % 16)]) * g,
                                               __uint_as_float(r[k / 16][2 * (k % 16) + 1]) * g);
                    }
                    store_box(&tm_out, box, w, p0, q0, p.P, p.Q, lane);
                }
                __syncwarp();
            }
        }
        if constexpr (!SWAP) store_box_finish(lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other's work may touch it
    if (warp == PAIR_MMA) {
        tc_fence_after();
        tmem_dealloc_2cta(tmem, TMEM_COLS);
    }
}

// Scale tiles [row blocks][chunks][512 bytes] in boxes of CHUNKS chunks of
// `blocks` row blocks; what lies outside reads as zero.
bool make_scale_map(CUtensorMap* m, const uint8_t* base, int64_t row_blocks, int64_t chunks, uint32_t blocks) {
    const uint64_t dims[3] = {128, (uint64_t)chunks, (uint64_t)row_blocks};
    const uint64_t strides[2] = {512, (uint64_t)chunks * 512};
    const uint32_t box[3] = {128, CHUNKS, blocks};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(base), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Codes [rows][K/2 bytes]: 128B-swizzled boxes of 128 bytes x box_rows; rows
// and bytes past the end read as zero codes.
bool make_rows_code_map(CUtensorMap* m, const uint8_t* base, int64_t rows, int64_t K, uint32_t box_rows) {
    const uint64_t dims[2] = {(uint64_t)K / 2, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)K / 2};
    const uint32_t box[2] = {128, box_rows};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int TN, bool SPLIT>
int launch_one(const GemmFp4Args& a, GemmParams& p, int split, int sms, cudaStream_t stream) {
    using C = Cfg<TN>;
    p.P = (int)a.N;
    p.Q = (int)a.M;
    p.sfp = a.w_scales;
    p.sfq = a.x_scales;
    p.p_tiles = (p.P + BP - 1) / BP;
    p.q_tiles = (p.Q + TN - 1) / TN;
    p.sfp_blocks = (p.P + 127) / 128;
    p.sfq_blocks = (p.Q + 127) / 128;
    CUtensorMap tp, tq;
    if (!make_rows_code_map(&tp, a.w_codes, p.P, a.K, BP) || !make_rows_code_map(&tq, a.x_codes, p.Q, a.K, TN))
        return FP4ATTN_ERR_CUDA;
    auto kernel = gemm_fp4_kernel<TN, SPLIT>;
    constexpr size_t smem = (size_t)C::STAGE * C::STAGES + 1024;
    static_assert(smem + sizeof(Bars) <= 227 * 1024, "shared memory budget");
    static_assert(!SPLIT || (size_t)TN * BP * 4 <= (size_t)C::STAGE * C::STAGES, "the parts fit the ring");
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    const long long tiles = (long long)p.p_tiles * p.q_tiles;
    const unsigned grid = (unsigned)(SPLIT ? tiles * split : (tiles < sms ? tiles : sms));
    return launch_behind(kernel, dim3(grid), THREADS, smem, stream, SPLIT ? split : 1, tp, tq, p) == cudaSuccess
               ? FP4ATTN_OK
               : FP4ATTN_ERR_CUDA;
}

template <bool SWAP>
int launch_pair(const GemmFp4Args& a, GemmParams& p, int sms, cudaStream_t stream) {
    using C = PairCfg;
    p.P = (int)(SWAP ? a.N : a.M);
    p.Q = (int)(SWAP ? a.M : a.N);
    p.p_tiles = (p.P + PAIR_TILE - 1) / PAIR_TILE;
    p.q_tiles = (p.Q + PAIR_TILE - 1) / PAIR_TILE;
    CUtensorMap tp, tq, tsp, tsq, to;
    if (!make_rows_code_map(&tp, SWAP ? a.w_codes : a.x_codes, p.P, a.K, 128) ||
        !make_rows_code_map(&tq, SWAP ? a.x_codes : a.w_codes, p.Q, a.K, 128) ||
        !make_scale_map(&tsp, SWAP ? a.w_scales : a.x_scales, (p.P + 127) / 128, p.chunks, 1) ||
        !make_scale_map(&tsq, SWAP ? a.x_scales : a.w_scales, (p.Q + 127) / 128, p.chunks, 2))
        return FP4ATTN_ERR_CUDA;
    to = tp;  // not read with SWAP
    if (!SWAP && !make_store_map(&to, a.out, a.M, a.N, a.ld)) return FP4ATTN_ERR_CUDA;
    auto kernel = gemm_fp4_pair_kernel<SWAP>;
    constexpr size_t smem = (size_t)C::STAGE * C::STAGES + STORE_BYTES + 1024;
    static_assert(smem + sizeof(Bars) <= 227 * 1024, "shared memory budget");
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    const long long tiles = (long long)p.p_tiles * p.q_tiles, pairs = sms / 2;
    return launch_behind(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), PAIR_THREADS, smem, stream, 1, tp, tq,
                         tsp, tsq, to, p) == cudaSuccess
               ? FP4ATTN_OK
               : FP4ATTN_ERR_CUDA;
}

}  // namespace

int launch_gemm_fp4(const GemmFp4Args& a, cudaStream_t stream) {
    if (a.M == 0 || a.N == 0) return FP4ATTN_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    GemmParams p{};
    p.chunks = (int)scale_chunks(a.K);
    p.stages = (p.chunks + CHUNKS - 1) / CHUNKS;
    p.gx = a.gx;
    p.gw = a.gw;
    p.bias = a.bias;
    p.out = a.out;
    p.ld = a.ld;
    p.N = (int)a.N;
    p.weight_ready = a.weight_ready ? 1 : 0;
    p.status = a.status;
    // Tiles of 128 x 128.  More than one a SM: pairs, with x on the lanes where the
    // output's rows take bulk stores.  2048 x 2048 x 6144 (256 tiles): 15.3 us in
    // pairs, 24 on single CTAs; 1024 x 2048 x 6144 (128): 14.9 and 13.4.
    const int64_t tiles = (a.N + 127) / 128 * ((a.M + 127) / 128);
    if (a.M > 128 && tiles > sms)
        return (a.N & 7) == 0 && (a.ld & 7) == 0 ? launch_pair<false>(a, p, sms, stream)
                                                 : launch_pair<true>(a, p, sms, stream);
    // Few tiles: K split over a cluster, where that leaves enough of it for each
    // CTA and the clusters find room at once (8 of them at a time fit 64 SMs
    // easily, 128 not).  K = 6144, 2 to 16 tiles: 13 -> 9.3 us split by 8, 10.4 by
    // 4; K = 2080: 7.5 us whole, 9.5 split.  The join costs little for short x
    // only: split by two 8.7 instead of 11.8 us with 16 rows, 14.5 instead of 13.4
    // with 128.
    int split = 1;
    if (p.stages >= 16)
        split = tiles * 8 <= 96 ? 8 : tiles * 4 <= 128 ? 4 : tiles * 2 <= sms - 8 && a.M <= 64 ? 2 : 1;
    if (a.M <= 16) return split > 1 ? launch_one<16, true>(a, p, split, sms, stream) : launch_one<16, false>(a, p, 1, sms, stream);
    if (a.M <= 64) return split > 1 ? launch_one<64, true>(a, p, split, sms, stream) : launch_one<64, false>(a, p, 1, sms, stream);
    return split > 1 ? launch_one<128, true>(a, p, split, sms, stream) : launch_one<128, false>(a, p, 1, sms, stream);
}

}  // namespace fp4attn
