// Straight-through gradients of the NVFP4 linear layer:
//
//   dx = g_w dy W~       [M, K]      W~, X~: the unit-scale values s * e2m1 of
//   dw = g_x dy^T X~     [N, K]      the forward's operands, exact in bf16
//   dbias = column sums of dy
//
// The operands are expanded to bf16 once (a few percent of the products' time)
// and both products run in ONE persistent launch on the BF16 tensor cores:
//   * a CTA pair owns a 256 x TN tile (tcgen05 cta_group::2): each CTA loads
//     128 rows of one operand and half of the other's TN columns and keeps 128
//     rows of the accumulator.  A single CTA would read 12 KB of operands and
//     take in as many for 128 clocks of tensor work, more than its shared
//     memory passes; the pair needs 8 KB;
//   * W~ and X~ are taken as they lie: their contraction runs down the rows, so
//     they enter as MN-major tiles, and so does dy for dw.  Nothing is
//     transposed in memory.  One box shape (64 x 64, 128B swizzle) serves all;
//   * two accumulators fill TMEM, so the epilogue of a tile runs under the
//     products of the next;
//   * few tiles and a long contraction: a tile is split into parts, fp32 parts
//     meet in the workspace and a last launch adds them in order.
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
constexpr int PAIRS = 74;  // of 148 SMs

template <int TN>
struct Cfg {
    static constexpr uint32_t A_BYTES = 2 * PANEL;               // 128 rows (or columns) of A per CTA
    static constexpr uint32_t B_BYTES = (TN / 128) * PANEL;      // TN / 2 columns of B per CTA
    static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
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
    int split;        // parts of the contraction
    int units;        // row_tiles * col_tiles * split
    int a_mn;         // A is MN-major (dy^T)
    const float* g;
    __nv_bfloat16* out;
    long long ld;
    float* part;      // [split][rows][K] when split > 1
};

struct BwdGemmParams {
    Product prod[2];
    int K;            // output columns of both
    int col_tiles;
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
    int which, rt, ct, part, s_begin, s_end;
};
__device__ __forceinline__ Unit unit_of(const BwdGemmParams& p, int u) {
    Unit w;
    w.which = u >= p.prod[0].units;
    const Product& q = p.prod[w.which];
    const int v = w.which ? u - p.prod[0].units : u;
    const int tiles = q.row_tiles * p.col_tiles;
    w.part = v / tiles;
    tile_of(v - w.part * tiles, q.row_tiles, p.col_tiles, w.rt, w.ct);
    const int stages = (q.contraction + BKC - 1) / BKC;
    w.s_begin = (int)((long long)stages * w.part / q.split);
    w.s_end = (int)((long long)stages * (w.part + 1) / q.split);
    return w;
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
            const int col0 = TN * w.ct + TN / 2 * (int)rank;
            const CUtensorMap* tb = a_mn ? &tm_x : &tm_w;
            for (int ks = w.s_begin; ks < w.s_end; ++ks, ++it) {
                const int slot = it % C::STAGES;
                if (it >= C::STAGES &&
                    !warp_wait(smem_u32(&sm.empty[slot]), (it / C::STAGES - 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    // the pair's copies all count on the first CTA's barrier
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[slot]), 2 * C::STAGE);
                    const uint32_t full = mapa(smem_u32(&sm.full[slot]), 0);
                    const uint32_t at = ring_u + C::STAGE * slot;
                    const int k0 = BKC * ks;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_2d_2cta(at + PANEL * i, &tm_dy, a_mn ? row0 + 64 * i : k0, a_mn ? k0 : row0 + 64 * i,
                                         full);
#pragma unroll
                    for (int j = 0; j < TN / 128; ++j)
                        tma_load_2d_2cta(at + C::A_BYTES + PANEL * j, tb, col0 + 64 * j, k0, full);
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
            constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(TN >> 3) << 17) |
                                       ((uint32_t)(BM >> 4) << 24);
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, p.status, kLimitNs));
            };
            int it = 0, local = 0;
            bool ok = true;
            for (int u = pair; ok && u < units; u += pairs, ++local) {
                const Unit w = unit_of(p, u);
                const bool a_mn = p.prod[w.which].a_mn != 0;
                const uint32_t idesc = IDESC | (a_mn ? 1u << 15 : 0u);
                // K-major A: 8-row groups 1 KB apart, 16 values 32 bytes on.  MN-major: 64-column
                // panels PANEL apart, 8-row groups 1 KB apart, 16 rows 2 KB on
                const uint32_t a_lbo = a_mn ? PANEL : 16u;
                const uint64_t a_step = a_mn ? 2048u >> 4 : 32u >> 4;
                const uint32_t acc = tmem + (local & 1 ? 256u : 0u);
                if (local >= 2 && !wait(smem_u32(&sm.acc_empty[local & 1]), ((local >> 1) - 1) & 1)) break;
                tc_fence_after();
                for (int ks = w.s_begin; ks < w.s_end; ++ks, ++it) {
                    const int slot = it % C::STAGES;
                    if (!wait(smem_u32(&sm.full[slot]), (it / C::STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        tc_fence_after();
                        const uint32_t at = ring_u + C::STAGE * slot;
                        const uint64_t ad = smem_desc(at, a_lbo, 1024, LAYOUT_SW128);
                        const uint64_t bd = smem_desc(at + C::A_BYTES, PANEL, 1024, LAYOUT_SW128);
#pragma unroll
                        for (int k = 0; k < BKC / 16; ++k)
                            mma_bf16_ss_2cta(acc, ad + a_step * k, bd + (2048u >> 4) * k, idesc,
                                             (ks > w.s_begin || k > 0) ? 1u : 0u);
                        tc_commit_2cta(smem_u32(&sm.empty[slot]));
                        if (ks == w.s_end - 1) tc_commit_2cta(smem_u32(&sm.acc_full[local & 1]));
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
        // a warp reads its quarter of the lanes and half of the columns, 64 at a time
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t box = ring_u + C::STAGES * C::STAGE + STORE_BOX * warp;
        int local = 0;
        for (int u = pair; u < units; u += pairs, ++local) {
            const Unit w = unit_of(p, u);
            const Product& q = p.prod[w.which];
            const uint32_t acc = tmem + lanes + (local & 1 ? 256u : 0u);
            if (!warp_wait(smem_u32(&sm.acc_full[local & 1]), (local >> 1) & 1, abort_flag, p.status)) break;
            tc_fence_after();
            const float g = q.g ? __ldg(q.g) : 1.0f;
            if (u == 0 && threadIdx.x == 0 && rank == 0) {
                const float g1 = p.prod[1].g ? __ldg(p.prod[1].g) : 1.0f;
                if (bad_gscale(g) || bad_gscale(g1)) raise_status(p.status, FP4ATTN_ERR_RANGE);
            }
            const int row0 = BM * w.rt + 128 * (int)rank + 32 * quarter, row = row0 + lane;
#pragma unroll 1
            for (int i = 0; i < TN / 128; ++i) {
                const int c0 = TN / 2 * half + 64 * i, col = TN * w.ct + c0;
                uint32_t r[2][32];
                tmem_ld32(acc + c0, r[0]);
                tmem_ld32(acc + c0 + 32, r[1]);
                tmem_wait_ld();
                if (i == TN / 128 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&sm.acc_empty[local & 1]), 0));
                }
                if (q.split > 1) {
                    // K is a multiple of 32
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (row < q.rows && col + 32 * h < p.K && FP4ATTN_IN_BOUNDS(w.part < q.split, p.status)) {
                            float4* dst =
                                reinterpret_cast<float4*>(q.part + ((long long)w.part * q.rows + row) * p.K + col + 32 * h);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                dst[k] = make_float4(__uint_as_float(r[h][4 * k]), __uint_as_float(r[h][4 * k + 1]),
                                                     __uint_as_float(r[h][4 * k + 2]), __uint_as_float(r[h][4 * k + 3]));
                        }
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

// out = g * (sum of the parts, in order), eight columns per thread.
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ BwdGemmParams p) {
    pdl_wait();
    pdl_trigger();
    const long long per_row = p.K / 8;
    const long long n0 = p.prod[0].split > 1 ? p.prod[0].rows * per_row : 0;
    const long long n1 = p.prod[1].split > 1 ? p.prod[1].rows * per_row : 0;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n0 + n1; i += (long long)gridDim.x * 256) {
        const Product& q = p.prod[i >= n0];
        const long long j = i >= n0 ? i - n0 : i;
        const long long row = j / per_row, col = 8 * (j - row * per_row);
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int k = 0; k < q.split; ++k) {
            const float4* src = reinterpret_cast<const float4*>(q.part + ((long long)k * q.rows + row) * p.K + col);
            const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
            s[0] += lo.x, s[1] += lo.y, s[2] += lo.z, s[3] += lo.w;
            s[4] += hi.x, s[5] += hi.y, s[6] += hi.z, s[7] += hi.w;
        }
        const float g = q.g ? __ldg(q.g) : 1.0f;
        if (FP4ATTN_IN_BOUNDS(row < q.rows, p.status))
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

struct Plan {
    int tn;
    int split[2];  // dw, dx
};

// Tile width and splits by a model of the launch in clocks: units go round the
// pairs, the products with the longer contraction first.
Plan make_plan(int64_t M, int64_t N, int64_t K, bool want_dw, bool want_dx) {
    Plan best{256, {1, 1}};
    double best_cost = -1.0;
    const int64_t rows[2] = {want_dw ? N : 0, want_dx ? M : 0}, contraction[2] = {M, N};
    static const int splits[8] = {1, 2, 3, 4, 6, 8, 12, 16};
    for (int tn = 256; tn >= 128; tn -= 128) {
        const double per_stage = tn == 256 ? 512.0 : 288.0, per_unit = 1500.0;
        const int64_t ct = (K + tn - 1) / tn;
        int64_t tiles[2], stages[2];
        for (int i = 0; i < 2; ++i) {
            tiles[i] = (rows[i] + BM - 1) / BM * ct;
            stages[i] = (contraction[i] + BKC - 1) / BKC;
        }
        const bool may_split = tiles[0] + tiles[1] < 2 * PAIRS;
        for (int a = 0; a < (may_split ? 8 : 1); ++a) {
            for (int b = 0; b < (may_split ? 8 : 1); ++b) {
                const int s[2] = {splits[a], splits[b]};
                if ((a && (s[0] * 2 > stages[0] || !tiles[0])) || (b && (s[1] * 2 > stages[1] || !tiles[1]))) continue;
                double unit[2], join = 0.0;
                int64_t n[2];
                for (int i = 0; i < 2; ++i) {
                    unit[i] = (double)((stages[i] + s[i] - 1) / s[i]) * per_stage + per_unit;
                    n[i] = tiles[i] * s[i];
                    if (s[i] > 1) join += 4000.0 + (double)s[i] * rows[i] * K * 8.0 / 4000.0;
                }
                const int first = unit[0] >= unit[1] ? 0 : 1;
                const int64_t n0 = (n[first] + PAIRS - 1) / PAIRS, all = (n[0] + n[1] + PAIRS - 1) / PAIRS;
                const double cost = (double)n0 * unit[first] + (double)(all - n0) * unit[1 - first] + join;
                if (best_cost < 0.0 || cost < best_cost) {
                    best_cost = cost;
                    best.tn = tn;
                    best.split[0] = s[0];
                    best.split[1] = s[1];
                }
            }
        }
    }
    return best;
}

int64_t part_floats(const Plan& pl, int64_t M, int64_t N, int64_t K, bool want_dw, bool want_dx) {
    int64_t n = 0;
    if (want_dw && pl.split[0] > 1) n += pl.split[0] * N * K;
    if (want_dx && pl.split[1] > 1) n += pl.split[1] * M * K;
    return n;
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

size_t linear_backward_part_bytes(int64_t M, int64_t N, int64_t K) {
    int64_t most = 0;
    for (int want = 1; want < 4; ++want) {
        const bool dw = want & 1, dx = want & 2;
        const int64_t n = part_floats(make_plan(M, N, K, dw, dx), M, N, K, dw, dx);
        most = n > most ? n : most;
    }
    return (size_t)most * 4;
}

int launch_linear_backward(const LinearBwdArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    // the operands' unit-scale values
    if (a.dx && launch_dequant_rows(a.w_codes, a.w_scales, nullptr, a.N, a.K, a.w_bf16, false, stream) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    if (a.dw && launch_dequant_rows(a.x_codes, a.x_scales, nullptr, a.M, a.K, a.x_bf16, false, stream) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    if (a.dbias && launch_column_sums(a.dy, a.ld_dy, a.M, a.N, a.colsum_part, a.dbias, stream) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    if (!a.dx && !a.dw) return FP4ATTN_OK;
    const Plan pl = make_plan(a.M, a.N, a.K, a.dw != nullptr, a.dx != nullptr);
    BwdGemmParams p{};
    p.K = (int)a.K;
    p.col_tiles = (int)((a.K + pl.tn - 1) / pl.tn);
    p.status = a.status;
    float* part = a.part;
    Product prod[2]{};
    for (int i = 0; i < 2; ++i) {
        Product& q = prod[i];
        const bool dw = i == 0;
        q.rows = (int)(dw ? a.N : a.M);
        q.contraction = (int)(dw ? a.M : a.N);
        q.a_mn = dw ? 1 : 0;
        q.g = dw ? a.gx : a.gw;
        q.out = dw ? a.dw : a.dx;
        q.ld = dw ? a.K : a.ld_dx;
        q.split = pl.split[i];
        q.row_tiles = q.out ? (q.rows + BM - 1) / BM : 0;
        q.units = q.row_tiles * p.col_tiles * q.split;
        if (!q.out) q.split = 1;
        if (q.split > 1) {
            q.part = part;
            part += (long long)q.split * q.rows * a.K;
        }
    }
    const auto stages = [](const Product& q) { return (q.contraction + BKC - 1) / BKC / q.split; };
    const int first = (prod[0].units && (!prod[1].units || stages(prod[0]) >= stages(prod[1]))) ? 0 : 1;
    p.prod[0] = prod[first];
    p.prod[1] = prod[1 - first];
    CUtensorMap dy, w, x;
    if (!make_map(&dy, a.dy, a.M, a.N, a.ld_dy)) return FP4ATTN_ERR_CUDA;
    w = x = dy;
    if (a.dx && !make_map(&w, a.w_bf16, a.N, a.K, a.K)) return FP4ATTN_ERR_CUDA;
    if (a.dw && !make_map(&x, a.x_bf16, a.M, a.K, a.K)) return FP4ATTN_ERR_CUDA;
    CUtensorMap out[2] = {dy, dy};  // a split product, or an absent one, does not use its own
    for (int i = 0; i < 2; ++i)
        if (p.prod[i].units && !make_store_map(&out[i], p.prod[i].out, p.prod[i].rows, a.K, p.prod[i].ld))
            return FP4ATTN_ERR_CUDA;
    const int units = p.prod[0].units + p.prod[1].units;
    const int pairs = units < sms / 2 ? units : sms / 2;
    const int st = pl.tn == 256 ? launch_products<256>(p, dy, w, x, out, pairs, stream)
                                : launch_products<128>(p, dy, w, x, out, pairs, stream);
    if (st != FP4ATTN_OK) return st;
    if (p.prod[0].split > 1 || p.prod[1].split > 1) {
        long long n = 0;
        for (int i = 0; i < 2; ++i)
            if (p.prod[i].split > 1) n += (long long)p.prod[i].rows * (a.K / 8);
        const long long grid = (n + 255) / 256;
        if (launch_behind(join_parts_kernel, dim3((unsigned)(grid < 1184 ? grid : 1184)), 256, 0, stream, 1, p) != cudaSuccess)
            return FP4ATTN_ERR_CUDA;
    }
    return FP4ATTN_OK;
}

}  // namespace fp4attn
