// Straight-through gradients of the NVFP4 linear layer:
//
//   dx = g_w dy W~       [M, K]      W~, X~: the unit-scale values s * e2m1 of
//   dw = g_x dy^T X~     [N, K]      the forward's operands, exact in bf16
//   dbias = column sums of dy
//
// The operands are expanded to bf16 once, in a launch that also takes the partial
// column sums (50 us of 825 at 8192 x 6144 x 6144, mostly HBM), and both products
// run in ONE persistent launch on the BF16 tensor cores:
//   * a CTA pair owns a 256 x TN tile (tcgen05 cta_group::2): each CTA loads
//     128 rows of one operand and half of the other's TN columns and keeps 128
//     rows of the accumulators;
//   * what bounds large products is how fast L2 feeds the SMs (about 42 bytes a
//     clock each, 12 TB/s in all): a 256-column tile takes 64 bytes a clock of
//     tensor work, a 512-column one 48.  At 8192 x 6144 x 6144 the launch takes
//     753 us with 512 columns (1.64 PFLOP/s, the tensor pipe 92% busy; 820 us with
//     256, of which 665 remain when the loads are left out), and longer when the
//     power cap lowers the clock;
//   * W~ and X~ are taken as they lie: their contraction runs down the rows, so
//     they enter as MN-major tiles, and so does dy for dw.  Nothing is
//     transposed in memory.  One box shape (64 x 64, 128B swizzle) serves all;
//   * accumulators of 256 columns: narrow tiles take turns between the two that
//     TMEM holds, and the epilogue of one runs under the products of the next;
//     a 512-column tile takes both, and its first half is stored while the
//     second still waits for its last products;
//   * tiles may be split along the contraction (all of a small product's, or the
//     last ones, which do not fill a round of the pairs): fp32 parts meet in the
//     workspace and a last launch adds them in order.
// Every wait is bounded (FP4ATTN_ERR_TIMEOUT).
#include <cuda_bf16.h>

#include "nvfp4_rows.cuh"
#include "tile_store.cuh"

namespace fp4attn {

namespace {

constexpr int BM = 256;  // rows of a pair's tile
constexpr int BKC = 64;  // contraction per stage
constexpr int THREADS = 32 * (STORE_WARPS + 2);
constexpr int WARP_PRODUCER = STORE_WARPS, WARP_MMA = STORE_WARPS + 1;
constexpr uint32_t PANEL = 64 * 128;  // 64 rows of 64 bf16
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int PAIRS = 74;  // of 148 SMs; with fewer, plans made for these are slower, not wrong

template <int TN>
struct Cfg {
    static constexpr int N = TN < 256 ? TN : 256;            // columns of one accumulator
    static constexpr int HALVES = TN / N;                    // accumulators of a tile
    static constexpr uint32_t A_BYTES = 2 * PANEL;           // 128 rows (or columns) of A per CTA
    static constexpr uint32_t B_HALF = (N / 128) * PANEL;    // N / 2 columns of B per CTA
    static constexpr uint32_t STAGE = A_BYTES + HALVES * B_HALF;
    static constexpr int STAGES = (int)(193u * 1024 / STAGE) < 8 ? (int)(193u * 1024 / STAGE) : 8;
};

struct Bars {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t final_;
    uint32_t tmem_base;
    int abort_flag;
};

// One of the two products.
struct Product {
    int rows;         // rows of the output
    int contraction;
    int row_tiles;
    int whole;        // tiles done at once; the ones behind them are split
    int split;        // into parts of the contraction
    int units;        // whole + split * (tiles - whole)
    int a_mn;         // A is MN-major (dy^T)
    const float* g;
    __nv_bfloat16* out;
    long long ld;
    float* part;      // [tiles - whole][split][BM][TN]
};

struct BwdGemmParams {
    Product prod[2];
    int K;            // output columns of both
    int col_tiles, tn;
    // dbias: column sums of dy, from their parts
    const float* colsum_part;
    int colsum_parts, N;
    float* dbias;
    int* status;
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, kLimitNs));
}
__device__ __forceinline__ bool drain_wait(uint32_t bar, uint32_t parity) {
    int dummy = 0;
    return mbar_wait(bar, parity, &dummy, nullptr, kDrainNs);
}

// 256-row tiles in groups of 8, the group's column tiles outermost: a wave of
// 74 tiles reads about 8 + 9 operand strips.
constexpr int GROUP = 8;
__device__ __forceinline__ void tile_of(int t, int row_tiles, int col_tiles, int& rt, int& ct) {
    const int per = GROUP * col_tiles;
    const int grp = t / per, in = t - grp * per;
    const int rows = min(GROUP, row_tiles - grp * GROUP);
    ct = in / rows;
    rt = grp * GROUP + (in - ct * rows);
}

struct Unit {
    int which, rt, ct, s_begin, s_end;
    int part;  // index into the product's parts, -1 for a whole tile
};
__device__ __forceinline__ Unit unit_of(const BwdGemmParams& p, int u) {
    Unit w;
    w.which = u >= p.prod[0].units;
    const Product& q = p.prod[w.which];
    const int v = w.which ? u - p.prod[0].units : u;
    const int stages = (q.contraction + BKC - 1) / BKC;
    if (v < q.whole) {
        tile_of(v, q.row_tiles, p.col_tiles, w.rt, w.ct);
        w.part = -1;
        w.s_begin = 0;
        w.s_end = stages;
    } else {
        // the parts of a tile lie far apart: neighbours read the same contraction
        const int tail = q.row_tiles * p.col_tiles - q.whole;
        const int k = (v - q.whole) / tail, i = v - q.whole - k * tail;
        tile_of(q.whole + i, q.row_tiles, p.col_tiles, w.rt, w.ct);
        w.part = i * q.split + k;
        w.s_begin = (int)((long long)stages * k / q.split);
        w.s_end = (int)((long long)stages * (k + 1) / q.split);
    }
    return w;
}

// Which accumulator half h of a CTA's tile number `local` takes: tiles of 512
// columns take both, narrower ones take turns.  A tile that ends within its first
// half (the last of a row of them) has no second one.
template <int TN>
__device__ __forceinline__ int acc_of(int local, int h) { return TN > 256 ? h : local & 1; }
template <int TN>
__device__ __forceinline__ int halves_of(const BwdGemmParams& p, const Unit& w) {
    return TN > 256 && TN * w.ct + 256 < p.K ? 2 : 1;
}

template <int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    linear_bwd_kernel(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_out0,
                      const __grid_constant__ CUtensorMap tm_out1, const __grid_constant__ BwdGemmParams p) {
    using C = Cfg<TN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars sm;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_u = smem_u32(ring);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int units = p.prod[0].units + p.prod[1].units;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.acc_full[i]), 1);
            mbar_init(smem_u32(&sm.acc_empty[i]), 2 * STORE_WARPS);  // the epilogue warps of both CTAs
        }
        mbar_init(smem_u32(&sm.final_), 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc_2cta(smem_u32(&sm.tmem_base), 512);
        tmem_relinquish_2cta();
    }
    if (warp == WARP_PRODUCER && lane == 0) {
        prefetch_tmap(&tm_dy);
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort_flag = &sm.abort_flag;
    pdl_wait();
    pdl_trigger();

    if (warp == WARP_PRODUCER) {
        // ------------------------------------------------------ producer --
        int it = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const Unit w = unit_of(p, u);
            const bool a_mn = p.prod[w.which].a_mn != 0;
            const int row0 = BM * w.rt + 128 * (int)rank;
            const int col0 = TN * w.ct + C::N / 2 * (int)rank;
            const CUtensorMap* tb = a_mn ? &tm_x : &tm_w;
            const int halves = halves_of<TN>(p, w);
            for (int ks = w.s_begin; ks < w.s_end; ++ks, ++it) {
                const int slot = it % C::STAGES;
                if (it >= C::STAGES &&
                    !warp_wait(smem_u32(&sm.empty[slot]), (it / C::STAGES - 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    // the pair's copies all count on the first CTA's barrier
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[slot]), 2 * (C::A_BYTES + C::B_HALF * halves));
                    const uint32_t full = mapa(smem_u32(&sm.full[slot]), 0);
                    const uint32_t at = ring_u + C::STAGE * slot;
                    const int k0 = BKC * ks;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_2d_2cta(at + PANEL * i, &tm_dy, a_mn ? row0 + 64 * i : k0, a_mn ? k0 : row0 + 64 * i,
                                         full);
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
                        if (h < halves)
#pragma unroll
                            for (int j = 0; j < C::N / 128; ++j)
                                tma_load_2d_2cta(at + C::A_BYTES + C::B_HALF * h + PANEL * j, tb, col0 + C::N * h + 64 * j,
                                                 k0, full);
                }
                __syncwarp();
            }
        }
        if (rank == 0 && lane == 0 && *abort_flag)
            for (int i = (it > C::STAGES ? it - C::STAGES : 0); i < it; ++i)
                drain_wait(smem_u32(&sm.full[i % C::STAGES]), (i / C::STAGES) & 1);
    } else if (warp == WARP_MMA) {
        // ----------------------------------------------------------- MMA --
        if (rank == 0) {
            const bool leader = elect_one_sync();
            // kind::f16, fp32 accumulator, bf16 operands, B MN-major (1 << 16), M = 256
            constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(C::N >> 3) << 17) |
                                       ((uint32_t)(BM >> 4) << 24);
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, p.status, kLimitNs));
            };
            int it = 0, local = 0, uses[2] = {0, 0};  // of the accumulators, before this unit
            bool ok = true;
            for (int u = pair; ok && u < units; u += pairs, ++local) {
                const Unit w = unit_of(p, u);
                const int halves = halves_of<TN>(p, w);
                const bool a_mn = p.prod[w.which].a_mn != 0;
                const uint32_t idesc = IDESC | (a_mn ? 1u << 15 : 0u);
                // K-major A: 8-row groups 1 KB apart, 16 values 32 bytes on.  MN-major: 64-column
                // panels PANEL apart, 8-row groups 1 KB apart, 16 rows 2 KB on
                const uint32_t a_lbo = a_mn ? PANEL : 16u;
                const uint64_t a_step = a_mn ? 2048u >> 4 : 32u >> 4;
                for (int ks = w.s_begin; ok && ks < w.s_end; ++ks, ++it) {
                    const int slot = it % C::STAGES;
                    if (!wait(smem_u32(&sm.full[slot]), (it / C::STAGES) & 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h) {
                        if (h >= halves) break;
                        const int buf = acc_of<TN>(local, h), use = buf ? uses[1] : uses[0];
                        if (ks == w.s_begin && use > 0 && !wait(smem_u32(&sm.acc_empty[buf]), (use - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        if (leader) {
                            tc_fence_after();
                            const uint32_t at = ring_u + C::STAGE * slot;
                            const uint64_t ad = smem_desc(at, a_lbo, 1024, LAYOUT_SW128);
                            const uint64_t bd = smem_desc(at + C::A_BYTES + C::B_HALF * h, PANEL, 1024, LAYOUT_SW128);
#pragma unroll
                            for (int k = 0; k < BKC / 16; ++k)
                                mma_bf16_ss_2cta(tmem + 256u * buf, ad + a_step * k, bd + (2048u >> 4) * k, idesc,
                                                 (ks > w.s_begin || k > 0) ? 1u : 0u);
                            if (ks == w.s_end - 1) tc_commit_2cta(smem_u32(&sm.acc_full[buf]));
                            if (h == halves - 1) tc_commit_2cta(smem_u32(&sm.empty[slot]));
                        }
                        __syncwarp();
                    }
                }
                if (acc_of<TN>(local, 0) == 0 || halves == 2) ++uses[0];
                if (acc_of<TN>(local, 0) == 1 || halves == 2) ++uses[1];
            }
            if (leader) {
                tc_commit_2cta(smem_u32(&sm.final_));
                drain_wait(smem_u32(&sm.final_), 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------ epilogue --
        // a warp reads its quarter of the lanes and half of the columns, 64 at a time
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t box = ring_u + C::STAGES * C::STAGE + STORE_BOX * warp;
        int local = 0, uses[2] = {0, 0};
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs, ++local) {
            const Unit w = unit_of(p, u);
            const int halves = halves_of<TN>(p, w);
            const Product& q = p.prod[w.which];
            const float g = q.g ? __ldg(q.g) : 1.0f;
            if (u == 0 && threadIdx.x == 0 && rank == 0) {
                const float g1 = p.prod[1].g ? __ldg(p.prod[1].g) : 1.0f;
                if (bad_gscale(g) || bad_gscale(g1)) raise_status(p.status, FP4ATTN_ERR_RANGE);
            }
            const int in_tile = 128 * (int)rank + 32 * quarter, row0 = BM * w.rt + in_tile;
#pragma unroll 1
            for (int h = 0; h < halves; ++h) {
                const int buf = acc_of<TN>(local, h);
                if (!warp_wait(smem_u32(&sm.acc_full[buf]), (buf ? uses[1]++ : uses[0]++) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + lanes + 256u * buf;
#pragma unroll 1
                for (int i = 0; i < C::N / 128; ++i) {
                    const int c0 = C::N / 2 * half + 64 * i, in_col = C::N * h + c0, col = TN * w.ct + in_col;
                    uint32_t r[2][32];
                    tmem_ld32(acc + c0, r[0]);
                    tmem_ld32(acc + c0 + 32, r[1]);
                    tmem_wait_ld();
                    if (i == C::N / 128 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&sm.acc_empty[buf]), 0));
                    }
                    if (w.part >= 0) {
                        // fp32, the tile's whole rows: what lies past the matrix is never read
                        float4* dst = reinterpret_cast<float4*>(
                            q.part + ((long long)w.part * BM + in_tile + lane) * TN + in_col);
                        if (FP4ATTN_IN_BOUNDS(w.part < q.split * (q.row_tiles * p.col_tiles - q.whole), p.status))
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                dst[k] = make_float4(__uint_as_float(r[k / 8][4 * (k % 8)]),
                                                     __uint_as_float(r[k / 8][4 * (k % 8) + 1]),
                                                     __uint_as_float(r[k / 8][4 * (k % 8) + 2]),
                                                     __uint_as_float(r[k / 8][4 * (k % 8) + 3]));
                    } else {
                        uint32_t v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            v[k] = pack_bf16x2(__uint_as_float(r[k / 16][2 * (k % 16)]) * g,
                                               __uint_as_float(r[k / 16][2 * (k % 16) + 1]) * g);
                        store_box(w.which ? &tm_out1 : &tm_out0, box, v, row0, col, q.rows, p.K, lane);
                    }
                    __syncwarp();
                }
            }
        }
        store_box_finish(lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other's work may touch it
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc_2cta(tmem, 512);
    }
}

// The last launch: dbias = sum of the partial column sums, and the split tiles'
// out = g * (sum of the parts), all in order.  A CTA takes 2048 / tn rows of a
// tile at a time, a thread eight columns.
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ BwdGemmParams p, const int sum_blocks) {
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < sum_blocks) {
        // 64 columns by four shares of the parts, which meet in order
        __shared__ float sum[4][64];
        const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, c = blockIdx.x * 64 + tx;
        float s = 0.0f;
        if (c < p.N) {
            const int k0 = p.colsum_parts * ty / 4, k1 = p.colsum_parts * (ty + 1) / 4;
#pragma unroll 8
            for (int k = k0; k < k1; ++k) s += __ldcg(p.colsum_part + (long long)k * p.N + c);
        }
        sum[ty][tx] = s;
        __syncthreads();
        if (ty == 0 && c < p.N) p.dbias[c] = (sum[0][tx] + sum[1][tx]) + (sum[2][tx] + sum[3][tx]);
        return;
    }
    const int per_row = p.tn / 8, rows = 256 / per_row, groups = BM / rows;
    const int tail0 = p.prod[0].row_tiles * p.col_tiles - p.prod[0].whole;
    const int tail1 = p.prod[1].row_tiles * p.col_tiles - p.prod[1].whole;
    for (int b = (int)blockIdx.x - sum_blocks; b < (tail0 + tail1) * groups; b += (int)gridDim.x - sum_blocks) {
        const int t = b / groups;
        const Product& q = p.prod[t >= tail0];
        const int i = t >= tail0 ? t - tail0 : t;
        int rt, ct;
        tile_of(q.whole + i, q.row_tiles, p.col_tiles, rt, ct);
        const int in_row = (b - t * groups) * rows + (int)threadIdx.x / per_row, in_col = (int)threadIdx.x % per_row * 8;
        const int row = BM * rt + in_row, col = p.tn * ct + in_col;
        if (row >= q.rows || col >= p.K) continue;
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int k = 0; k < q.split; ++k) {
            const float4* src =
                reinterpret_cast<const float4*>(q.part + ((long long)(i * q.split + k) * BM + in_row) * p.tn + in_col);
            const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
            s[0] += lo.x, s[1] += lo.y, s[2] += lo.z, s[3] += lo.w;
            s[4] += hi.x, s[5] += hi.y, s[6] += hi.z, s[7] += hi.w;
        }
        const float g = q.g ? __ldg(q.g) : 1.0f;
        if (FP4ATTN_IN_BOUNDS(row < q.rows && col + 8 <= p.K, p.status))
            *reinterpret_cast<uint4*>(q.out + row * q.ld + col) =
                make_uint4(pack_bf16x2(g * s[0], g * s[1]), pack_bf16x2(g * s[2], g * s[3]),
                           pack_bf16x2(g * s[4], g * s[5]), pack_bf16x2(g * s[6], g * s[7]));
    }
}

// bf16 matrix [rows][cols], rows `ld` elements apart, in boxes of 64 x 64.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, 64};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tile width and splits by a model of the launch in clocks: units go round the
// pairs in order, the longer ones first, so a pair has the longest way to go that
// starts first.  Either product may be split (few tiles, a long contraction), and
// the last tiles of the second, which do not fill a round of the pairs any more.
// A stage costs what its bytes take (48, 32 or 24 KB at about 40 bytes a clock).
// An epilogue takes about 18 clocks a column and hides under the next unit's
// products unless the tile takes all of TMEM (512 columns: 30, with the pause of
// the loads); of a split tile, in fp32, twice that.  The plans are within ten percent of the best ones found at
// 3001 x 200 x 544, 1000 x 64 x 256, 4096 x 256 x 1024, 256 x 4096 x 4096 and 8192
// x 1024 x 1024 (M x N x K); with splits of small totals only, 28972 x 976 x 928
// took 231 us (now 131) and 100 x 15912 x 3328 142 (102).
LinearBwdPlan make_plan(int64_t M, int64_t N, int64_t K, bool want_dw, bool want_dx) {
    LinearBwdPlan best{};
    double best_cost = -1.0;
    const int64_t rows[2] = {want_dw ? N : 0, want_dx ? M : 0}, contraction[2] = {M, N};
    constexpr int MOST = 4;  // splits of 2^0 .. 2^MOST
    for (int tn = 512; tn >= 128; tn /= 2) {
        const double per_stage = tn == 512 ? 1300.0 : tn == 256 ? 780.0 : 585.0;
        const int64_t ct = (K + tn - 1) / tn;
        const double filled = tn == 512 && (K - 1) % 512 < 256 ? ((double)ct - 0.5) / (double)ct : 1.0;
        int64_t tiles[2], stages[2];
        double unit_cost[2][MOST + 1], join_cost[2][MOST + 1];
        int splits[2];
        auto unit = [&](int i, int split) {
            const double products = (double)((stages[i] + split - 1) / split) * per_stage;
            const double epilogue = (tn == 512 ? 30.0 : 18.0) * tn * (split > 1 ? 2.0 : 1.0);
            return tn == 512 ? (products + epilogue) * filled : (products > epilogue ? products : epilogue) + 1500.0;
        };
        auto join = [&](int64_t tail, int split) { return 5000.0 + (double)tail * split * (100.0 + BM * tn * 4.0 / 2500.0); };
        for (int i = 0; i < 2; ++i) {
            tiles[i] = (rows[i] + BM - 1) / BM * ct;
            stages[i] = (contraction[i] + BKC - 1) / BKC;
            splits[i] = 1;
            unit_cost[i][0] = unit(i, 1);
            join_cost[i][0] = 0.0;
            for (int k = 1; k <= MOST && tiles[i] && (tiles[i] << k) <= 4 * PAIRS && (2 << k) <= stages[i]; ++k) {
                unit_cost[i][k] = unit(i, 1 << k);
                join_cost[i][k] = join(tiles[i], 1 << k);
                splits[i] = k + 1;
            }
        }
        auto offer = [&](double cost, int64_t whole0, int64_t whole1, int split0, int split1, int first) {
            if (best_cost >= 0.0 && cost >= best_cost) return;
            best_cost = cost;
            best = LinearBwdPlan{tn, {tiles[0], tiles[1]}, {whole0, whole1}, {split0, split1}, first};
        };
        for (int a = 0; a < splits[0]; ++a) {
            for (int b = 0; b < splits[1]; ++b) {
                const int64_t n[2] = {tiles[0] << a, tiles[1] << b}, all = n[0] + n[1];
                const double u[2] = {unit_cost[0][a], unit_cost[1][b]}, joins = join_cost[0][a] + join_cost[1][b];
                const int f = (n[0] && (!n[1] || u[0] >= u[1])) ? 0 : 1;
                const int64_t head = (n[f] + PAIRS - 1) / PAIRS;
                auto way = [&](int64_t units) {  // of the pair with most to do, over the first `units`
                    const int64_t rounds = (units + PAIRS - 1) / PAIRS, h = head < rounds ? head : rounds;
                    return (double)h * u[f] + (double)(rounds - h) * u[1 - f];
                };
                const int64_t w0 = a ? 0 : tiles[0], w1 = b ? 0 : tiles[1];
                offer(joins + way(all), w0, w1, 1 << a, 1 << b, f);
                // the last tiles of the product that ends the launch, if it is whole
                const int last = n[1 - f] ? 1 - f : f;
                const int64_t rest = all % PAIRS;
                if ((last ? b : a) || !rest || rest > tiles[last] || all == rest) continue;
                int s = (int)(PAIRS / rest);
                if (s > 16) s = 16;
                if (s > stages[last] / 2) s = (int)(stages[last] / 2);
                if (s < 2) continue;
                const double extra = joins > 0.0 ? join(rest, s) - 5000.0 : join(rest, s);
                offer(joins + way(all - rest) + unit(last, s) + extra, last ? w0 : w0 - rest, last ? w1 - rest : w1,
                      last ? 1 << a : s, last ? s : 1 << b, f);
            }
        }
    }
    return best;
}

template <int TN>
int launch_products(const BwdGemmParams& p, const CUtensorMap& dy, const CUtensorMap& w, const CUtensorMap& x,
                    const CUtensorMap (&out)[2], int pairs, cudaStream_t stream) {
    using C = Cfg<TN>;
    constexpr size_t smem = (size_t)C::STAGE * C::STAGES + STORE_BYTES + 1024;
    static_assert(smem + sizeof(Bars) <= 227 * 1024, "shared memory budget");
    auto kernel = linear_bwd_kernel<TN>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    return launch_behind(kernel, dim3(2 * pairs), THREADS, smem, stream, 1, dy, w, x, out[0], out[1], p) == cudaSuccess
               ? FP4ATTN_OK
               : FP4ATTN_ERR_CUDA;
}

}  // namespace

LinearBwdPlan linear_backward_plan(int64_t M, int64_t N, int64_t K, bool want_dw, bool want_dx) {
    return make_plan(M, N, K, want_dw, want_dx);
}

size_t linear_backward_part_bytes(const LinearBwdPlan& pl) {
    return (size_t)((pl.tiles[0] - pl.whole[0]) * pl.split[0] + (pl.tiles[1] - pl.whole[1]) * pl.split[1]) * BM * pl.tn * 4;
}

int launch_linear_backward(const LinearBwdArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    int colsum_parts = 0;
    if (launch_backward_prepare(a, colsum_parts, stream) != cudaSuccess) return FP4ATTN_ERR_CUDA;
    const LinearBwdPlan& pl = a.plan;
    BwdGemmParams p{};
    p.K = (int)a.K;
    p.tn = pl.tn;
    p.col_tiles = (int)((a.K + pl.tn - 1) / pl.tn);
    p.colsum_part = a.colsum_part;
    p.colsum_parts = colsum_parts;
    p.N = (int)a.N;
    p.dbias = a.dbias;
    p.status = a.status;
    float* part = a.part;
    int tail = 0;
    for (int i = 0; i < 2; ++i) {
        Product& q = p.prod[i == pl.first ? 0 : 1];
        const bool dw = i == 0;
        q.rows = (int)(dw ? a.N : a.M);
        q.contraction = (int)(dw ? a.M : a.N);
        q.a_mn = dw ? 1 : 0;
        q.out = dw ? a.dw : a.dx;
        q.g = !q.out ? nullptr : dw ? a.gx : a.gw;  // an absent product's scale is not read
        q.ld = dw ? a.K : a.ld_dx;
        q.row_tiles = q.out ? (q.rows + BM - 1) / BM : 0;
        q.whole = (int)pl.whole[i];
        q.split = pl.split[i];
        const int split_tiles = (int)(pl.tiles[i] - pl.whole[i]);
        q.units = q.whole + split_tiles * q.split;
        q.part = part;
        part += (long long)split_tiles * q.split * BM * pl.tn;
        tail += split_tiles;
    }
    if (a.dx || a.dw) {
        CUtensorMap dy, w, x;
        if (!make_map(&dy, a.dy, a.M, a.N, a.ld_dy)) return FP4ATTN_ERR_CUDA;
        w = x = dy;
        if (a.dx && !make_map(&w, a.w_bf16, a.N, a.K, a.K)) return FP4ATTN_ERR_CUDA;
        if (a.dw && !make_map(&x, a.x_bf16, a.M, a.K, a.K)) return FP4ATTN_ERR_CUDA;
        CUtensorMap out[2] = {dy, dy};  // an absent product does not use its own
        for (int i = 0; i < 2; ++i)
            if (p.prod[i].units && !make_store_map(&out[i], p.prod[i].out, p.prod[i].rows, a.K, p.prod[i].ld))
                return FP4ATTN_ERR_CUDA;
        const int units = p.prod[0].units + p.prod[1].units;
        const int pairs = units < sms / 2 ? units : sms / 2;
        const int st = pl.tn == 512   ? launch_products<512>(p, dy, w, x, out, pairs, stream)
                       : pl.tn == 256 ? launch_products<256>(p, dy, w, x, out, pairs, stream)
                                      : launch_products<128>(p, dy, w, x, out, pairs, stream);
        if (st != FP4ATTN_OK) return st;
    }
    const int sum_blocks = a.dbias ? (int)((a.N + 63) / 64) : 0;
    int blocks = tail * pl.tn / 8;  // 2048 / tn rows at a time
    blocks = blocks < 1184 ? blocks : 1184;
    if (sum_blocks + blocks > 0 && launch_behind(join_parts_kernel, dim3((unsigned)(sum_blocks + blocks)), 256, 0, stream, 1, p,
                                                 sum_blocks) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    return FP4ATTN_OK;
}

}  // namespace fp4attn
