// The two norms around a block's branch, with its gate, its residual and the
// modulation of the next one, and their gradients:
//
//   y = x + gate * (post_weight * norm(h))
//   z = norm(y) * pre_weight * (1 + scale) + shift
//   norm(v) = v / sqrt(mean(v^2) + eps), or the same of v - mean(v)
//
// (DiT blocks: Peebles and Xie, "Scalable Diffusion Models with Transformers",
// 2023; a norm on the branch's output as well: Ding et al., "CogView", 2021.)
// Both directions are bound by HBM: every row is read once and written once.
// What it takes to get there is few instructions per value and enough bytes on
// their way at any time:
//   * A team of warps holds a row in registers, up to 24 values a thread; the teams of a CTA (one per SM) take turns down a range of
//     rows.  Products of the per-channel vectors (gate post_weight, pre_weight (1
//     + scale), shift) are made once per range and sample, in shared memory; the
//     backward's sums down the columns stay in registers over the range.  Rows
//     too wide for a CTA are shared by a cluster.
//   * The rows ahead come in by bulk copies into a ring in shared memory, one
//     ring per team, so loads stay in flight through reductions and stores.
//   * Two reductions over the team per row, for the layer norm too: its
//     variance is taken about a pivot (the mean of eight values of the row; for
//     y, of x) together with the mean, and again about that mean in the rare
//     row whose pivot lay more than a standard deviation off, where the
//     difference of squares would lose bits.
// The forward's z can leave as NVFP4 rows (rounded to bf16 first, as the
// quantiser of a bf16 z would see it), so that the next linear layer reads
// 9/16 byte a value instead of writing, reading and quantising 2-byte ones.
// The CTAs' column sums meet in the workspace and are added in order: no atomics,
// equal calls give equal bits.
//
// Forward 109568 x 6144, fp32 residual: 1.37 ms, 5.9 TB/s; backward 36864 x 6144:
// bf16 458 us (5.9 TB/s), layer norm 547, fp32 618 (6.6 TB/s).  What is left in
// the bf16 layer norms, quantised ones above all (36864 x 6144: 377 us, 226 at
// HBM's rate), is instructions: 57% of the issue slots, the rest latency.
#include <type_traits>

#include <cuda_bf16.h>

#include "nvfp4_rows.cuh"

namespace fp4attn {

namespace {

constexpr int MAX_COLS = 6144;  // of a CTA
constexpr int FWD_THREADS = 512;
constexpr uint64_t kLimitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int MAX_SLOTS = 6;
constexpr int MAX_CLUSTER = 3;  // 16384 channels

// ---------------------------------------------------------------- teams --

// A unit is what a thread loads at once: 8 values of bf16 rows, 4 of fp32 rows
// (16 bytes of the residual either way, so that its stores fill whole sectors).
template <int U>
using Packed = std::conditional_t<U == 8, uint4, uint2>;

__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[4]) {
    v[0] = pair_of(w.x), v[1] = pair_of(w.y), v[2] = pair_of(w.z), v[3] = pair_of(w.w);
}
__device__ __forceinline__ void unpack(uint2 w, float2 (&v)[2]) { v[0] = pair_of(w.x), v[1] = pair_of(w.y); }
__device__ __forceinline__ uint32_t pack_pair(float2 v) { return pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ uint4 pack(const float2 (&v)[4]) {
    return make_uint4(pack_pair(v[0]), pack_pair(v[1]), pack_pair(v[2]), pack_pair(v[3]));
}
__device__ __forceinline__ uint2 pack(const float2 (&v)[2]) { return make_uint2(pack_pair(v[0]), pack_pair(v[1])); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Residual units in shared or global memory.
__device__ __forceinline__ void load_res(const void* row, int u, float2 (&v)[4]) {
    unpack(static_cast<const uint4*>(row)[u], v);
}
__device__ __forceinline__ void load_res(const void* row, int u, float2 (&v)[2]) {
    const float4 f = static_cast<const float4*>(row)[u];
    v[0] = make_float2(f.x, f.y), v[1] = make_float2(f.z, f.w);
}
__device__ __forceinline__ void store_res(void* row, int u, const float2 (&v)[4]) { static_cast<uint4*>(row)[u] = pack(v); }
__device__ __forceinline__ void store_res(void* row, int u, const float2 (&v)[2]) {
    static_cast<float4*>(row)[u] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
// The values of a unit of a bf16 vector, or `absent` for a null one.
template <int U>
__device__ __forceinline__ void load_vector(const __nv_bfloat16* p, int64_t at, float absent, float2 (&v)[U / 2]) {
    if (p) {
        unpack(__ldg(reinterpret_cast<const Packed<U>*>(p + at)), v);
    } else {
#pragma unroll
        for (int i = 0; i < U / 2; ++i) v[i] = both(absent);
    }
}

// What a thread knows of its team: TPR threads of the CTA, or (WIDE) of each CTA of
// the cluster.  Sums of up to MAX_K quantities.  A wide team's warps write their
// sums into every CTA and arrive on a barrier there: several teams of a cluster
// go their own ways, and a row costs no barrier over all of it.
template <int TPR, int MAX_K, bool WIDE>
struct Team {
    static constexpr int warps = TPR / 32;
    static constexpr int MAX_WARPS = (warps + 3) / 4 * 4 * (WIDE ? MAX_CLUSTER : 1);
    // floats per team, zeroed: two buffers that alternate
    static constexpr int SCRATCH = warps == 1 && !WIDE ? 4 : 2 * MAX_K * MAX_WARPS;
    float* scratch;
    int index, phase;
    uint32_t rank, ranks;
    // WIDE: this team's barrier (ranks * warps arrivals), and what a wait needs
    uint32_t bar, parity;
    volatile int* abort_flag;
    int* status;

    // WIDE, behind the lanes' remote stores
    __device__ __forceinline__ void arrive_and_wait() {
        __syncwarp();
        const int lane = threadIdx.x & 31;
        if (lane < (int)ranks) mbar_arrive_cluster(mapa(bar, (uint32_t)lane));
        mbar_wait_cluster(bar, parity, abort_flag, status, kLimitNs);
        parity ^= 1;
    }

    __device__ __forceinline__ void sync() {
        if constexpr (WIDE)
            arrive_and_wait();
        else if constexpr (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "n"(TPR) : "memory");
    }

    // Sums over the team of K values a thread, the same bits in every thread.
    // Ends every use that the threads made of shared memory before it.
    template <int K>
    __device__ __forceinline__ void sum(float (&v)[K]) {
        static_assert(K <= MAX_K, "scratch");
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if constexpr (!WIDE && warps == 1) {
            __syncwarp();
        } else {
            float* at = scratch + phase * (MAX_K * MAX_WARPS);
            phase ^= 1;
            const int warp = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
            if constexpr (WIDE) {
                if (lane < (int)ranks) {
                    const uint32_t base = mapa(smem_u32(at), (uint32_t)lane);
#pragma unroll
                    for (int k = 0; k < K; ++k) st_cluster(base + 4u * (k * MAX_WARPS + rank * warps + warp), v[k]);
                }
            } else if (lane == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) at[k * MAX_WARPS + warp] = v[k];
            }
            sync();
            // what lies past the last warp is zero
            const int n = WIDE ? warps * (int)ranks : MAX_WARPS;
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < (WIDE ? n : MAX_WARPS); w += 4)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float4 f = *reinterpret_cast<const float4*>(at + k * MAX_WARPS + w);
                    v[k] += (f.x + f.y) + (f.z + f.w);
                }
        }
    }
};

// The columns of a CTA: all of them, or a share of whole 64-channel chunks.
__device__ __forceinline__ int first_column(int cols_per_cta, uint32_t rank) { return cols_per_cta * (int)rank; }

// Mean of eight neighbouring values in the middle of the row (of this CTA's
// columns): of a residual (8: bf16, 4: fp32) or (2) of bf16 values in fours.
template <int KIND>
__device__ __forceinline__ float pivot_of(const void* row, int units) {
    float2 s;
    if constexpr (KIND == 8) {
        float2 v[4];
        load_res(row, units >> 1, v);
        s = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    } else {
        float2 v[2], w[2];
        const int u = units >> 1;  // an even number of units: eight channels make two
        if constexpr (KIND == 4) {
            load_res(row, u - 1, v);
            load_res(row, u, w);
        } else {
            unpack(static_cast<const uint2*>(row)[u - 1], v);
            unpack(static_cast<const uint2*>(row)[u], w);
        }
        s = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(w[0], w[1]));
    }
    return 0.125f * (s.x + s.y);
}
// The same pivot for every CTA of a cluster.
template <int TPR, int MAX_K, bool WIDE>
__device__ __forceinline__ void share_pivots(Team<TPR, MAX_K, WIDE>& team, float& p, float& q) {
    if constexpr (WIDE) {
        float v[2] = {threadIdx.x == 0 ? p : 0.0f, threadIdx.x == 0 ? q : 0.0f};
        team.sum(v);
        p = v[0] / (float)team.ranks;
        q = v[1] / (float)team.ranks;
    }
}

// ------------------------------------------------------------- forward --
//
// The products of the vectors (A = gate post_weight, B = pre_weight
// (1 + scale), S = shift) stand in shared memory, shared by the CTA's teams,
// which take turns down the rows of one sample after another; that leaves
// registers for 512 threads, twice the warps of the backward to hide the
// reductions and the quantiser behind.

template <int TPR, int J, int U, bool LAYER, bool QUANT, bool WIDE>
__global__ void __launch_bounds__(FWD_THREADS, 1) norm_gate_kernel(const __grid_constant__ NormArgs a) {
    constexpr int TEAMS = FWD_THREADS / TPR, ES = U == 4 ? 4 : 2, P = U / 2;
    using TeamT = Team<TPR, 2, WIDE>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[TEAMS * MAX_SLOTS];
    __shared__ __align__(16) float scratch[TEAMS * TeamT::SCRATCH];
    __shared__ uint64_t team_bars[TEAMS];
    __shared__ int abort_all;
    __shared__ ScaleTable table;  // not used (and not there) unless QUANT
    const int t = threadIdx.x % TPR;
    TeamT team;
    team.index = threadIdx.x / TPR;
    team.scratch = scratch + team.index * TeamT::SCRATCH;
    team.phase = 0;
    team.rank = WIDE ? cluster_ctarank() : 0;
    team.ranks = WIDE ? cluster_nctarank() : 1;
    team.bar = smem_u32(&team_bars[team.index]);
    team.parity = 0;
    team.abort_flag = &abort_all;
    team.status = a.status;
    const int c0 = first_column(a.cols, team.rank), cols = min(a.cols, a.C - c0), NU = cols / U;
    pdl_wait();
    pdl_trigger();
    const float gz = QUANT ? (a.gz ? __ldg(a.gz) : 1.0f) : 1.0f;
    if (QUANT) make_scale_table(table, gz, threadIdx.x);
    if (threadIdx.x == 0) abort_all = 0;
    for (int i = threadIdx.x; i < TEAMS * MAX_SLOTS; i += blockDim.x) mbar_init(smem_u32(&bars[i]), 1);
    for (int i = threadIdx.x; i < (int)(sizeof(scratch) / 4); i += blockDim.x) scratch[i] = 0.0f;
    if (WIDE && threadIdx.x < TEAMS) mbar_init(smem_u32(&team_bars[threadIdx.x]), team.ranks * TeamT::warps);
    fence_mbar_init();
    __syncthreads();
    if constexpr (WIDE) cluster_sync();
    volatile int* abort_flag = &abort_all;
    const float guess = QUANT ? table.guess : 0.0f;
    if (QUANT && blockIdx.x == 0 && threadIdx.x == 0 && bad_gscale(gz)) raise_status(a.status, FP4ATTN_ERR_RANGE);

    const bool has_h = a.h != nullptr;
    const uint32_t x_bytes = (uint32_t)cols * ES, h_bytes = has_h ? (uint32_t)cols * 2 : 0;
    // four channels of each of A, B and S per entry: a unit of eight takes one from
    // either half, so that the threads of a warp read consecutive entries
    float4* vectors = reinterpret_cast<float4*>(smem);
    const int plane = a.cols / U;  // entries; A, B, S of U / 4 planes each
    const uint8_t* ring = smem + (size_t)12 * a.cols + (size_t)team.index * a.slots * a.slot_bytes;
    const uint32_t ring_u = smem_u32(ring), bars_u = smem_u32(&bars[team.index * MAX_SLOTS]);
    const int64_t clusters = gridDim.x / team.ranks, cluster = blockIdx.x / team.ranks;
    const int64_t r0 = a.rows * cluster / clusters, r1 = a.rows * (cluster + 1) / clusters;
    // thread 0's rows ahead: r0 + index, + TEAMS, ...
    int ahead = (int)((r1 - r0 - team.index + TEAMS - 1) / TEAMS);
    const uint8_t* x_next = static_cast<const uint8_t*>(a.x) + ((r0 + team.index) * a.ldx + c0) * ES;
    const __nv_bfloat16* h_next = a.h + ((r0 + team.index) * a.ldh + c0);
    const int64_t x_step = (int64_t)TEAMS * a.ldx * ES, h_step = (int64_t)TEAMS * a.ldh;
    auto fill = [&](int slot) {
        const uint32_t bar = bars_u + 8u * slot, at = ring_u + a.slot_bytes * slot;
        mbar_arrive_expect_tx(bar, x_bytes + h_bytes);
        bulk_load(at, x_next, x_bytes, bar);
        if (has_h) bulk_load(at + x_bytes, h_next, h_bytes, bar);
        x_next += x_step;
        h_next += h_step;
        --ahead;
    };
    if (t == 0)
        for (int s = 0; s < a.slots && ahead > 0; ++s) fill(s);
    const float inv_c = 1.0f / (float)a.C;
    const int sf_shift = 8 * ((t * U / 16) & 3);  // TPR U channels are whole chunks of 64

    bool finite = true;
    int slot = 0;
    uint32_t parity = 0;
    int64_t row = r0 + team.index;
    for (int64_t group = r0 / a.rows_per_group; group * a.rows_per_group < r1; ++group) {
        __syncthreads();
        for (int u = threadIdx.x; u < NU; u += blockDim.x) {
            const int64_t c = c0 + U * u;
            float2 p[P], q[P];
            auto put = [&](int which) {
#pragma unroll
                for (int k = 0; k < U / 4; ++k)
                    vectors[(which * (U / 4) + k) * plane + u] = make_float4(p[2 * k].x, p[2 * k].y, p[2 * k + 1].x, p[2 * k + 1].y);
            };
            load_vector<U>(a.gate, group * a.lgate + c, 1.0f, p);
            load_vector<U>(a.post, c, 1.0f, q);
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = __fmul2_rn(p[i], q[i]);
            put(0);
            load_vector<U>(a.pre, c, 1.0f, p);
            load_vector<U>(a.scale, group * a.lscale + c, 0.0f, q);
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = __ffma2_rn(p[i], q[i], p[i]);
            put(1);
            load_vector<U>(a.shift, group * a.lshift + c, 0.0f, p);
            put(2);
        }
        __syncthreads();
        auto vector = [&](int which, int u, float2(&v)[P]) {
#pragma unroll
            for (int k = 0; k < U / 4; ++k) {
                const float4 f = vectors[(which * (U / 4) + k) * plane + u];
                v[2 * k] = make_float2(f.x, f.y);
                v[2 * k + 1] = make_float2(f.z, f.w);
            }
        };
        const int64_t end = min((group + 1) * a.rows_per_group, r1);
        for (; row < end; row += TEAMS) {
            const bool ok = mbar_wait(bars_u + 8u * slot, parity, abort_flag, a.status, kLimitNs);
            const uint8_t* at = ring + (size_t)a.slot_bytes * slot;
            // the pivots of y (a guess from x) and h; channels past the row's end
            // hold them and add nothing
            float p = 0.0f, q = 0.0f;
            if (LAYER) {
                p = pivot_of<U>(at, NU);
                if (has_h) q = pivot_of<U == 8 ? 8 : 2>(at + x_bytes, NU);
                share_pivots(team, p, q);
            }
            const uint32_t q_word = pack_bf16x2(q, q);
            if (LAYER) q = bf16lo(q_word);
            float2 y[J][P];
            Packed<U> h[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + TPR * j;
                if (u < NU) {
                    load_res(at, u, y[j]);
                    if (has_h) h[j] = reinterpret_cast<const Packed<U>*>(at + x_bytes)[u];
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) y[j][i] = both(p);
                    if constexpr (U == 8)
                        h[j] = make_uint4(q_word, q_word, q_word, q_word);
                    else
                        h[j] = make_uint2(q_word, q_word);
                }
            }
            // a row that never came (its wait ran out) must not pass for one
            if (!ok) y[0][0].x = __int_as_float(0x7FC00000);
            if (has_h) {
                float r, mean_h = 0.0f;
                if constexpr (!LAYER) {
                    float2 s2 = both(0.0f);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        float2 f[P];
                        unpack(h[j], f);
#pragma unroll
                        for (int i = 0; i < P; ++i) s2 = __ffma2_rn(f[i], f[i], s2);
                    }
                    float s[1] = {s2.x + s2.y};
                    team.sum(s);
                    r = rsqrtf(__fmaf_rn(s[0], inv_c, a.eps));
                } else {
                    auto moments = [&](float pivot, bool all, float& d) {
                        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            float2 f[P];
                            unpack(h[j], f);
                            if (all || t + TPR * j < NU)
#pragma unroll
                                for (int i = 0; i < P; ++i) {
                                    f[i] = __fadd2_rn(f[i], both(-pivot));
                                    s1 = __fadd2_rn(s1, f[i]);
                                    s2 = __ffma2_rn(f[i], f[i], s2);
                                }
                        }
                        float s[2] = {s1.x + s1.y, s2.x + s2.y};
                        team.sum(s);
                        d = s[0] * inv_c;
                        return __fmaf_rn(-d, d, s[1] * inv_c);
                    };
                    float d, var = moments(q, true, d);
                    mean_h = q + d;
                    if (!(d * d <= var)) {
                        var = moments(mean_h, false, d);
                        mean_h += d;
                    }
                    r = rsqrtf(fmaxf(var, 0.0f) + a.eps);
                }
                // (h - mean) r as h r - mean r: its rounding is of the size of the mean's own
                const float2 r2 = both(r), mr2 = both(-mean_h * r);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (t + TPR * j < NU) {
                        float2 f[P], A[P];
                        unpack(h[j], f);
                        vector(0, t + TPR * j, A);
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            y[j][i] = __ffma2_rn(A[i], LAYER ? __ffma2_rn(f[i], r2, mr2) : __fmul2_rn(f[i], r2), y[j][i]);
                    }
                }
            } else {
                team.sync();
            }
            // every thread has its row: the slot is free
            if (t == 0 && ahead > 0 && !*abort_flag) fill(slot);
            if (++slot == a.slots) {
                slot = 0;
                parity ^= 1;
            }
            if (a.y) {
                void* y_at = static_cast<uint8_t*>(a.y) + (row * a.ldy + c0) * ES;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int u = t + TPR * j;
                    if (u < NU && FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status)) store_res(y_at, u, y[j]);
                }
            }
            if (!QUANT && !a.z) continue;
            float r, mr = 0.0f;  // norm(y) = y r + mr
            if constexpr (!LAYER) {
                float2 s2 = both(0.0f);
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < P; ++i) s2 = __ffma2_rn(y[j][i], y[j][i], s2);
                float s[1] = {s2.x + s2.y};
                team.sum(s);
                r = rsqrtf(__fmaf_rn(s[0], inv_c, a.eps));
            } else {
                auto moments = [&](float pivot, bool all, float& d) {
                    float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        if (all || t + TPR * j < NU)
#pragma unroll
                            for (int i = 0; i < P; ++i) {
                                const float2 f = __fadd2_rn(y[j][i], both(-pivot));
                                s1 = __fadd2_rn(s1, f);
                                s2 = __ffma2_rn(f, f, s2);
                            }
                    float s[2] = {s1.x + s1.y, s2.x + s2.y};
                    team.sum(s);
                    d = s[0] * inv_c;
                    return __fmaf_rn(-d, d, s[1] * inv_c);
                };
                float d, var = moments(p, true, d);
                p += d;
                if (!(d * d <= var)) {
                    var = moments(p, false, d);
                    p += d;
                }
                r = rsqrtf(fmaxf(var, 0.0f) + a.eps);
                mr = -p * r;
            }
            __nv_bfloat16* z_at = a.z + (row * a.ldz + c0);
            uint8_t* codes_at = a.codes + (row * a.C + c0) / 2;
            // where the scales of this row's first chunk go; a chunk is 128 words on
            uint32_t* scales_at = reinterpret_cast<uint32_t*>(a.scales) + ((row >> 7) * a.chunks + c0 / 64) * 128 +
                                  scale_word_in_tile((uint32_t)row & 127);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + TPR * j;
                float2 z[P];
                if (u < NU) {
                    float2 B[P], S[P];
                    vector(1, u, B);
                    vector(2, u, S);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        z[i] = __ffma2_rn(
                            LAYER ? __ffma2_rn(y[j][i], both(r), both(mr)) : __fmul2_rn(y[j][i], both(r)), B[i], S[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) z[i] = both(0.0f);
                }
                const Packed<U> w = pack(z);
                const bool on = u < NU && FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status);
                if constexpr (!QUANT) {
                    if (on) reinterpret_cast<Packed<U>*>(z_at)[u] = w;
                } else {
                    // 16 / U lanes share a block, 64 / U a word of four scales
                    unpack(w, z);
                    uint32_t m2 = amax_pair(w);
#pragma unroll
                    for (int o = 1; o < 16 / U; o *= 2) m2 = max_pair(m2, __shfl_xor_sync(0xffffffffu, m2, o));
                    const float m = max_nan(bf16lo(m2), bf16hi(m2));
                    finite = finite && (m < INFINITY);
                    uint32_t s8;
                    float inv;
                    row_block_scale(table, guess, m, gz, s8, inv);
#pragma unroll
                    for (int i = 0; i < P; ++i) z[i] = __fmul2_rn(z[i], both(inv));
                    if constexpr (U == 8) {
                        const uint32_t c = cvt_e2m1x8(z[0].x, z[0].y, z[1].x, z[1].y, z[2].x, z[2].y, z[3].x, z[3].y);
                        if (on) reinterpret_cast<uint32_t*>(codes_at)[u] = c;
                    } else {
                        const uint32_t c = cvt_e2m1x8(z[0].x, z[0].y, z[1].x, z[1].y, 0.0f, 0.0f, 0.0f, 0.0f);
                        if (on) reinterpret_cast<uint16_t*>(codes_at)[u] = (uint16_t)c;
                    }
                    uint32_t word = s8 << sf_shift;
#pragma unroll
                    for (int o = 16 / U; o < 64 / U; o *= 2) word |= __shfl_xor_sync(0xffffffffu, word, o);
                    if (on && t % (64 / U) == 0 &&
                        FP4ATTN_IN_BOUNDS(((row >> 7) * a.chunks + (c0 + U * u) / 64) * 512 + 512 <= scale_tile_bytes(a.rows, a.C),
                                          a.status))
                        scales_at[U * u / 64 * 128] = word;
                }
            }
        }
    }
    if (QUANT && !finite) raise_status(a.status, FP4ATTN_ERR_RANGE);
    if (t == 0 && *abort_flag) {
        // this team's own copies land before it leaves (bounded)
        int dummy = 0;
        for (int s = 0; s < a.slots; ++s)
            for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(bars_u + 8u * s, ph, &dummy, nullptr, kDrainNs);
    }
    if constexpr (WIDE) cluster_sync();  // no CTA leaves while another may write into it
}

// ------------------------------------------------------------ backward --
//
// With n = norm(y) = r (y - mean), dn = dz pre (1 + scale):
//   dx = dy + r (dn - n mean(dn n) - [layer] mean(dn))
// and with m = norm(h), dm = dx gate post:
//   dh = r_h (dm - m mean(dm m) - [layer] mean(dm))
// Sums down the rows of a sample: dz, dz n, dx m, in registers over a CTA's
// range of rows of one sample (an item), then over its teams in order.  A row is
// read from its slot twice (y and dy need not stay in registers in between).

template <int THREADS, int TPR, int J, int U, bool LAYER, bool WIDE>
__global__ void __launch_bounds__(THREADS, 1) norm_gate_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
    constexpr int TEAMS = THREADS / TPR, ES = U == 4 ? 4 : 2, P = U / 2;
    // 255 registers hold the vectors as well: 36864 x 6144, bf16: 476 -> 452 us (fp32
    // rows, whose loads take more of them: 625 -> 666)
    constexpr bool HELD = THREADS == 256 && U == 8;
    using TeamT = Team<TPR, 6, WIDE>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[TEAMS * MAX_SLOTS];
    __shared__ __align__(16) float scratch[TEAMS * TeamT::SCRATCH];
    __shared__ uint64_t team_bars[TEAMS];
    __shared__ int abort_all;
    const int t = threadIdx.x % TPR;
    TeamT team;
    team.index = threadIdx.x / TPR;
    team.scratch = scratch + team.index * TeamT::SCRATCH;
    team.phase = 0;
    team.rank = WIDE ? cluster_ctarank() : 0;
    team.ranks = WIDE ? cluster_nctarank() : 1;
    team.bar = smem_u32(&team_bars[team.index]);
    team.parity = 0;
    team.abort_flag = &abort_all;
    team.status = a.status;
    const int c0 = first_column(a.cols, team.rank), cols = min(a.cols, a.C - c0), NU = cols / U;
    if (threadIdx.x == 0) abort_all = 0;
    for (int i = threadIdx.x; i < TEAMS * MAX_SLOTS; i += blockDim.x) mbar_init(smem_u32(&bars[i]), 1);
    for (int i = threadIdx.x; i < (int)(sizeof(scratch) / 4); i += blockDim.x) scratch[i] = 0.0f;
    if (WIDE && threadIdx.x < TEAMS) mbar_init(smem_u32(&team_bars[threadIdx.x]), team.ranks * TeamT::warps);
    fence_mbar_init();
    __syncthreads();
    if constexpr (WIDE) cluster_sync();
    volatile int* abort_flag = &abort_all;
    pdl_wait();
    pdl_trigger();

    const bool has_h = a.h != nullptr, has_dy = a.dy != nullptr;
    const uint32_t res_bytes = (uint32_t)cols * ES, half_bytes = (uint32_t)cols * 2;
    // a slot: y, dy (residual type), dz, h (bf16)
    const uint32_t at_dy = res_bytes, at_dz = at_dy + (has_dy ? res_bytes : 0), at_h = at_dz + half_bytes;
    const uint32_t row_bytes = at_h + (has_h ? half_bytes : 0);
    // shared memory: A = gate post_weight and B = pre_weight (1 + scale), four
    // channels an entry (see the forward); where teams meet; the rings
    float4* vectors = reinterpret_cast<float4*>(smem);
    const int plane = a.cols / U;
    float* meet = reinterpret_cast<float*>(smem + (size_t)8 * a.cols);
    const uint8_t* ring = smem + (size_t)(TEAMS > 1 ? 20 : 8) * a.cols + (size_t)team.index * a.slots * a.slot_bytes;
    const uint32_t ring_u = smem_u32(ring), bars_u = smem_u32(&bars[team.index * MAX_SLOTS]);
    const int64_t clusters = gridDim.x / team.ranks, first_item = blockIdx.x / team.ranks;
    const int64_t items = a.groups * a.parts;
    auto item_rows = [&](int64_t item, int64_t& begin, int64_t& end) {
        const int64_t g = item / a.parts, p = item - g * a.parts;
        begin = g * a.rows_per_group + a.rows_per_group * p / a.parts;
        end = g * a.rows_per_group + a.rows_per_group * (p + 1) / a.parts;
    };
    // thread 0's rows ahead, over the CTA's items: of an item, `left` and where the next one lies
    int64_t ahead_item = first_item;
    int left = 0;
    const uint8_t *y_next = nullptr, *dy_next = nullptr;
    const __nv_bfloat16 *dz_next = nullptr, *h_next = nullptr;
    const int64_t y_step = (int64_t)TEAMS * a.ldy * ES, dy_step = (int64_t)TEAMS * a.lddy * ES,
                  dz_step = (int64_t)TEAMS * a.lddz, h_step = (int64_t)TEAMS * a.ldh;
    auto seek = [&]() {  // from a new item on to one that has a row for this team
        for (; ahead_item < items; ahead_item += clusters) {
            int64_t begin, end;
            item_rows(ahead_item, begin, end);
            begin += team.index;
            if (begin >= end) continue;
            left = (int)((end - begin + TEAMS - 1) / TEAMS);
            y_next = static_cast<const uint8_t*>(a.y) + (begin * a.ldy + c0) * ES;
            dy_next = static_cast<const uint8_t*>(a.dy) + (begin * a.lddy + c0) * ES;
            dz_next = a.dz + (begin * a.lddz + c0);
            h_next = a.h + (begin * a.ldh + c0);
            return;
        }
    };
    auto fill_next = [&](int slot) {
        if (left == 0) return;  // no item any more
        const uint32_t bar = bars_u + 8u * slot, at = ring_u + a.slot_bytes * slot;
        mbar_arrive_expect_tx(bar, row_bytes);
        bulk_load(at, y_next, res_bytes, bar);
        if (has_dy) bulk_load(at + at_dy, dy_next, res_bytes, bar);
        bulk_load(at + at_dz, dz_next, half_bytes, bar);
        if (has_h) bulk_load(at + at_h, h_next, half_bytes, bar);
        y_next += y_step;
        dy_next += dy_step;
        dz_next += dz_step;
        h_next += h_step;
        if (--left == 0) {
            ahead_item += clusters;
            seek();
        }
    };
    if (t == 0) {
        seek();
        for (int s = 0; s < a.slots; ++s) fill_next(s);
    }
    const float inv_c = 1.0f / (float)a.C;
    int slot = 0;
    uint32_t parity = 0;
    auto vector = [&](int which, int u, float2(&v)[P]) {
#pragma unroll
        for (int k = 0; k < U / 4; ++k) {
            const float4 f = vectors[(which * (U / 4) + k) * plane + u];
            v[2 * k] = make_float2(f.x, f.y);
            v[2 * k + 1] = make_float2(f.z, f.w);
        }
    };
    for (int64_t item = first_item; item < items; item += clusters) {
        int64_t begin, end;
        item_rows(item, begin, end);
        const int64_t group = item / a.parts;
        __syncthreads();
        for (int u = threadIdx.x; u < NU; u += blockDim.x) {
            const int64_t c = c0 + U * u;
            float2 p[P], q[P];
            auto put = [&](int which) {
#pragma unroll
                for (int k = 0; k < U / 4; ++k)
                    vectors[(which * (U / 4) + k) * plane + u] = make_float4(p[2 * k].x, p[2 * k].y, p[2 * k + 1].x, p[2 * k + 1].y);
            };
            load_vector<U>(a.gate, group * a.lgate + c, 1.0f, p);
            load_vector<U>(a.post, c, 1.0f, q);
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = __fmul2_rn(p[i], q[i]);
            put(0);
            load_vector<U>(a.pre, c, 1.0f, p);
            load_vector<U>(a.scale, group * a.lscale + c, 0.0f, q);
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = __ffma2_rn(p[i], q[i], p[i]);
            put(1);
        }
        __syncthreads();
        float2 s_dz[J][P], s_dzn[J][P], s_dxm[J][P], held_A[J][P], held_B[J][P];
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int i = 0; i < P; ++i) s_dz[j][i] = s_dzn[j][i] = s_dxm[j][i] = both(0.0f);
            if (HELD) {
                const int u = min(t + TPR * j, NU - 1);
                vector(0, u, held_A[j]);
                vector(1, u, held_B[j]);
            }
        }
        auto gate_of = [&](int j, int u, float2(&v)[P]) {
            if constexpr (HELD) {
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = held_A[j][i];
            } else {
                vector(0, u, v);
            }
        };
        auto pre_of = [&](int j, int u, float2(&v)[P]) {
            if constexpr (HELD) {
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = held_B[j][i];
            } else {
                vector(1, u, v);
            }
        };
        for (int64_t row = begin + team.index; row < end; row += TEAMS) {
            const bool ok = mbar_wait(bars_u + 8u * slot, parity, abort_flag, a.status, kLimitNs);
            const uint8_t* at = ring + (size_t)a.slot_bytes * slot;
            Packed<U> dz[J], h[J];
            float p = 0.0f, q = 0.0f;
            if (LAYER) {
                p = pivot_of<U>(at, NU);
                if (has_h) q = pivot_of<U == 8 ? 8 : 2>(at + at_h, NU);
                share_pivots(team, p, q);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + TPR * j;
                dz[j] = Packed<U>{};
                h[j] = Packed<U>{};
                if (u < NU) {
                    dz[j] = reinterpret_cast<const Packed<U>*>(at + at_dz)[u];
                    if (has_h) h[j] = reinterpret_cast<const Packed<U>*>(at + at_h)[u];
                }
            }
            float ry, rh, mean_y = 0.0f, mean_h = 0.0f, mean_dn = 0.0f, c1;
            // sums about the pivots p of y and q of h; whether those were near enough
            auto moments = [&]() -> bool {
                float2 s_y = both(0.0f), s_y2 = both(0.0f), s_dn = both(0.0f), s_dny = both(0.0f), s_h = both(0.0f),
                       s_h2 = both(0.0f);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int u = t + TPR * j;
                    if (u < NU) {
                        float2 y[P], d[P], f[P], B[P];
                        load_res(at, u, y);
                        if (!ok) y[0].x = __int_as_float(0x7FC00000);  // a row that never came
                        unpack(dz[j], d);
                        unpack(h[j], f);
                        pre_of(j, u, B);
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            d[i] = __fmul2_rn(d[i], B[i]);
                            if constexpr (LAYER) {
                                y[i] = __fadd2_rn(y[i], both(-p));
                                f[i] = __fadd2_rn(f[i], both(-q));
                                s_y = __fadd2_rn(s_y, y[i]);
                                s_h = __fadd2_rn(s_h, f[i]);
                                s_dn = __fadd2_rn(s_dn, d[i]);
                            }
                            s_y2 = __ffma2_rn(y[i], y[i], s_y2);
                            s_dny = __ffma2_rn(d[i], y[i], s_dny);
                            s_h2 = __ffma2_rn(f[i], f[i], s_h2);
                        }
                    }
                }
                if constexpr (!LAYER) {
                    float s[3] = {s_y2.x + s_y2.y, s_dny.x + s_dny.y, s_h2.x + s_h2.y};
                    team.sum(s);
                    ry = rsqrtf(__fmaf_rn(s[0], inv_c, a.eps));
                    rh = rsqrtf(__fmaf_rn(s[2], inv_c, a.eps));
                    c1 = s[1] * inv_c * ry;  // mean(dn n)
                    return true;
                } else {
                    float s[6] = {s_y.x + s_y.y, s_y2.x + s_y2.y, s_dn.x + s_dn.y, s_dny.x + s_dny.y, s_h.x + s_h.y,
                                  s_h2.x + s_h2.y};
                    team.sum(s);
                    const float d = s[0] * inv_c, e = s[4] * inv_c;
                    const float vy = __fmaf_rn(-d, d, s[1] * inv_c), vh = __fmaf_rn(-e, e, s[5] * inv_c);
                    mean_y = p + d;
                    mean_h = q + e;
                    mean_dn = s[2] * inv_c;
                    ry = rsqrtf(fmaxf(vy, 0.0f) + a.eps);
                    rh = rsqrtf(fmaxf(vh, 0.0f) + a.eps);
                    c1 = (s[3] * inv_c - d * mean_dn) * ry;
                    return d * d <= vy && e * e <= vh;
                }
            };
            if (!moments()) {
                p = mean_y;
                q = mean_h;
                moments();
            }
            // n = y r - mean r and the like: the products' roundings are of the size
            // of the mean's own.  dx = dy + r dn - r c1 n - r mean(dn)
            float2 dm[J][P];
            float2 s_dmm = both(0.0f), s_dm = both(0.0f);
            const float2 ry2 = both(ry), rh2 = both(rh), my2 = both(-mean_y * ry), mh2 = both(-mean_h * rh),
                         c12 = both(-c1 * ry), md2 = both(-mean_dn * ry);
            uint8_t* dx_at = static_cast<uint8_t*>(a.dx) + (row * a.lddx + c0) * ES;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + TPR * j;
                if (u < NU) {
                    float2 y[P], d[P], f[P], g[P], A[P], B[P];
                    load_res(at, u, y);
                    if (has_dy) {
                        load_res(at + at_dy, u, g);
                    } else {
#pragma unroll
                        for (int i = 0; i < P; ++i) g[i] = both(0.0f);
                    }
                    unpack(dz[j], d);
                    unpack(h[j], f);
                    gate_of(j, u, A);
                    pre_of(j, u, B);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 n = LAYER ? __ffma2_rn(y[i], ry2, my2) : __fmul2_rn(y[i], ry2);
                        const float2 m = LAYER ? __ffma2_rn(f[i], rh2, mh2) : __fmul2_rn(f[i], rh2);
                        s_dz[j][i] = __fadd2_rn(s_dz[j][i], d[i]);
                        s_dzn[j][i] = __ffma2_rn(d[i], n, s_dzn[j][i]);
                        if (LAYER) g[i] = __fadd2_rn(g[i], md2);
                        g[i] = __ffma2_rn(n, c12, g[i]);
                        g[i] = __ffma2_rn(__fmul2_rn(d[i], B[i]), ry2, g[i]);  // dx
                        s_dxm[j][i] = __ffma2_rn(g[i], m, s_dxm[j][i]);
                        dm[j][i] = __fmul2_rn(g[i], A[i]);
                        s_dmm = __ffma2_rn(dm[j][i], m, s_dmm);
                        if (LAYER) s_dm = __fadd2_rn(s_dm, dm[j][i]);
                    }
                    if (FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status)) store_res(dx_at, u, g);
                }
            }
            float k1 = 0.0f, k0 = 0.0f;  // dh = r dm + k1 h + k0
            if (!has_h) {
                team.sync();
            } else if constexpr (LAYER) {
                float s[2] = {s_dmm.x + s_dmm.y, s_dm.x + s_dm.y};
                team.sum(s);
                k1 = -rh * rh * (s[0] * inv_c);
                k0 = -k1 * mean_h - rh * (s[1] * inv_c);
            } else {
                float s[1] = {s_dmm.x + s_dmm.y};
                team.sum(s);
                k1 = -rh * rh * (s[0] * inv_c);
            }
            // no thread reads the slot any more
            if (t == 0 && !*abort_flag) fill_next(slot);
            if (++slot == a.slots) {
                slot = 0;
                parity ^= 1;
            }
            if (!has_h) continue;
            const float2 k12 = both(k1), k02 = both(k0);
            __nv_bfloat16* dh_at = a.dh + (row * a.lddh + c0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + TPR * j;
                if (u < NU) {
                    float2 f[P];
                    unpack(h[j], f);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        f[i] = __ffma2_rn(dm[j][i], rh2, LAYER ? __ffma2_rn(f[i], k12, k02) : __fmul2_rn(f[i], k12));
                    if (FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status))
                        reinterpret_cast<Packed<U>*>(dh_at)[u] = pack(f);
                }
            }
        }
        // the teams' sums, one team after the other; the last one writes them out
        float* part = a.part + item * 3 * (int64_t)a.C + c0;
        for (int k = 0; k < TEAMS; ++k) {
            if (team.index == k) {
                const bool last = k == TEAMS - 1;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int u = t + TPR * j;
                    if (u < NU && FP4ATTN_IN_BOUNDS(item < items, a.status)) {
#pragma unroll
                        for (int w = 0; w < 3; ++w) {
                            const float2(&v)[P] = w == 0 ? s_dz[j] : w == 1 ? s_dzn[j] : s_dxm[j];
#pragma unroll
                            for (int i = 0; i < P; i += 2) {
                                float4 f = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
                                float4* const m = reinterpret_cast<float4*>(meet + w * cols + U * u + 2 * i);
                                if (k > 0) {
                                    const float4 o = *m;
                                    f = make_float4(o.x + f.x, o.y + f.y, o.z + f.z, o.w + f.w);
                                }
                                if (last)
                                    *reinterpret_cast<float4*>(part + w * (int64_t)a.C + U * u + 2 * i) = f;
                                else
                                    *m = f;
                            }
                        }
                    }
                }
            }
            if (k < TEAMS - 1) __syncthreads();
        }
    }
    if (t == 0 && *abort_flag) {
        int dummy = 0;
        for (int s = 0; s < a.slots; ++s)
            for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(bars_u + 8u * s, ph, &dummy, nullptr, kDrainNs);
    }
    if constexpr (WIDE) cluster_sync();  // no CTA leaves while another may write into it
}

// Adds a sample's parts in order (32 columns by 8 shares of the parts per CTA;
// the shares meet in order) and makes the gradients of its vectors.  With one
// sample the weights' gradients follow at once; with more the sums are kept,
// in the first part's place, for norm_weights_kernel.
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormBwdArgs a) {
    __shared__ float sum[3][8][32];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t blocks = (a.C + 31) / 32;
    const int64_t g = blockIdx.x / blocks, c = (blockIdx.x - g * blocks) * 32 + tx;
    float* base = a.part + g * a.parts * 3 * (int64_t)a.C;
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (c < a.C) {
        const int p0 = (int)(a.parts * ty / 8), p1 = (int)(a.parts * (ty + 1) / 8);
#pragma unroll 4
        for (int p = p0; p < p1; ++p)
#pragma unroll
            for (int k = 0; k < 3; ++k) s[k] += __ldcg(base + ((int64_t)p * 3 + k) * a.C + c);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k][ty][tx] = s[k];
    __syncthreads();
    if (ty != 0 || c >= a.C) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s[k] += sum[k][w][tx];
    }
    const float post = a.post ? __bfloat162float(a.post[c]) : 1.0f, pre = a.pre ? __bfloat162float(a.pre[c]) : 1.0f;
    const int64_t at = g * (int64_t)a.C + c;
    if (a.dshift) a.dshift[at] = s[0];
    if (a.dscale) a.dscale[at] = s[1] * pre;
    if (a.dgate) a.dgate[at] = s[2] * post;
    if (a.groups > 1) {
        base[a.C + c] = s[1];
        base[2 * (int64_t)a.C + c] = s[2];
    } else {
        if (a.dpre) a.dpre[c] = s[1] * (1.0f + (a.scale ? __bfloat162float(a.scale[c]) : 0.0f));
        if (a.dpost) a.dpost[c] = s[2] * (a.gate ? __bfloat162float(a.gate[c]) : 1.0f);
    }
}

__global__ void __launch_bounds__(256) norm_weights_kernel(const __grid_constant__ NormBwdArgs a) {
    __shared__ float sum[2][8][32];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float s[2] = {0.0f, 0.0f};
    if (c < a.C) {
        const int64_t g0 = a.groups * ty / 8, g1 = a.groups * (ty + 1) / 8;
        for (int64_t g = g0; g < g1; ++g) {
            const float* base = a.part + g * a.parts * 3 * (int64_t)a.C;
            const float sc = a.scale ? __bfloat162float(a.scale[g * a.lscale + c]) : 0.0f;
            const float ga = a.gate ? __bfloat162float(a.gate[g * a.lgate + c]) : 1.0f;
            s[0] = __fmaf_rn(__ldcg(base + a.C + c), 1.0f + sc, s[0]);
            s[1] = __fmaf_rn(__ldcg(base + 2 * (int64_t)a.C + c), ga, s[1]);
        }
    }
    sum[0][ty][tx] = s[0];
    sum[1][ty][tx] = s[1];
    __syncthreads();
    if (ty != 0 || c >= a.C) return;
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        s[0] += sum[0][w][tx];
        s[1] += sum[1][w][tx];
    }
    if (a.dpre) a.dpre[c] = s[0];
    if (a.dpost) a.dpost[c] = s[1];
}

constexpr size_t SMEM_BYTES = 221 * 1024;  // of the vectors and rings
static_assert((8 + 2 * 12) * (size_t)MAX_COLS <= SMEM_BYTES && (20 + 4 * 12) * (size_t)(MAX_COLS / 2) <= SMEM_BYTES,
              "two slots of the widest rows");
static_assert((12 + 2 * 2 * 6) * (size_t)MAX_COLS <= SMEM_BYTES, "two slots of the forward's two widest teams");

// How rows of C channels are shared out: CTAs of a cluster, channels, threads
// and teams of a CTA, threads of a team, values a thread in eights.
struct Split {
    int ctas, cols, threads, teams, tpr, j8;
};
void share_columns(Split& s, int64_t C) {
    s.ctas = (int)((C + MAX_COLS - 1) / MAX_COLS);
    s.cols = s.ctas == 1 ? (int)C : (int)((C + 64 * s.ctas - 1) / (64 * s.ctas) * 64);
}
// Forward: up to 24 values a thread, teams of 32 to 256.
Split forward_split(int64_t C) {
    Split s{};
    share_columns(s, C);
    for (s.tpr = s.ctas > 1 ? 256 : 32; s.tpr * 24 < s.cols;) s.tpr *= 2;
    s.j8 = s.tpr == 32 || s.tpr == 256 ? (s.cols + 8 * s.tpr - 1) / (8 * s.tpr) : 3;
    if (s.tpr == 256 && (s.j8 < 2 || s.ctas > 1)) s.j8 = s.ctas > 1 ? 3 : 2;
    s.teams = FWD_THREADS / s.tpr;
    s.threads = s.teams * s.tpr;
    return s;
}
// Backward: narrow rows 16 values a thread and 384 threads of 168 registers,
// wide ones 24 and 256 of 255.  100000 x 512: 121 us the first way, 138 the
// second; 36864 x 6144, layer norm: 664 and 617.
Split backward_split(int64_t C) {
    Split s{};
    share_columns(s, C);
    if (s.ctas == 1 && s.cols <= 192 * 16) {
        static const int teams_of[5] = {32, 64, 96, 128, 192};
        int i = 0;
        while (teams_of[i] * 16 < s.cols) ++i;
        s.tpr = teams_of[i];
        s.j8 = s.cols <= 256 ? 1 : 2;
        s.threads = 384;
        s.teams = s.threads / s.tpr;
    } else {
        s.tpr = s.threads = 256;
        s.j8 = s.ctas == 1 && s.cols <= 256 * 16 ? 2 : 3;
        s.teams = 1;
    }
    return s;
}

// A launch on the device's SMs: clusters that fit at once, ring slots and
// shared memory.  Every field is set, or the status returned.
struct Shape {
    unsigned grid;
    int slots;
    size_t smem;
};
int shape_of(const void* kernel, const Split& s, size_t fixed_bytes, size_t slot_bytes, int64_t work, Shape& sh) {
    sh.slots = (int)((SMEM_BYTES - fixed_bytes) / (slot_bytes * s.teams));
    sh.slots = sh.slots < 1 ? 1 : sh.slots > MAX_SLOTS ? MAX_SLOTS : sh.slots;
    sh.smem = fixed_bytes + slot_bytes * s.teams * sh.slots;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sh.smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    int64_t clusters = sms / s.ctas;
    if (s.ctas > 1) {
        // not every SM finds a place in a cluster: a launch of more would go in two turns
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(clusters * s.ctas));
        cfg.blockDim = dim3((unsigned)s.threads);
        cfg.dynamicSmemBytes = sh.smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)s.ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) return FP4ATTN_ERR_CUDA;
        clusters = clusters < fit ? clusters : fit;
    }
    clusters = clusters < work ? clusters : work;
    sh.grid = (unsigned)(clusters * s.ctas);
    return FP4ATTN_OK;
}

template <typename Args>
int launch(void (*kernel)(Args), const Args& a, const Split& s, const Shape& sh, cudaStream_t stream) {
    return launch_behind(kernel, dim3(sh.grid), (unsigned)s.threads, sh.smem, stream, (unsigned)s.ctas, a) == cudaSuccess
               ? FP4ATTN_OK
               : FP4ATTN_ERR_CUDA;
}

using FwdKernel = void (*)(const NormArgs);
using BwdKernel = void (*)(const NormBwdArgs);

template <int TPR, int J8, bool WIDE>
FwdKernel fwd_of(bool f32, bool layer, bool quant) {
    if (f32) {
        if (layer)
            return quant ? norm_gate_kernel<TPR, 2 * J8, 4, true, true, WIDE> : norm_gate_kernel<TPR, 2 * J8, 4, true, false, WIDE>;
        return quant ? norm_gate_kernel<TPR, 2 * J8, 4, false, true, WIDE> : norm_gate_kernel<TPR, 2 * J8, 4, false, false, WIDE>;
    }
    if (layer) return quant ? norm_gate_kernel<TPR, J8, 8, true, true, WIDE> : norm_gate_kernel<TPR, J8, 8, true, false, WIDE>;
    return quant ? norm_gate_kernel<TPR, J8, 8, false, true, WIDE> : norm_gate_kernel<TPR, J8, 8, false, false, WIDE>;
}
FwdKernel forward_kernel(const Split& s, bool f32, bool layer, bool quant) {
    if (s.ctas > 1) return fwd_of<256, 3, true>(f32, layer, quant);
    switch (s.tpr) {
        case 32:
            return s.j8 == 1   ? fwd_of<32, 1, false>(f32, layer, quant)
                   : s.j8 == 2 ? fwd_of<32, 2, false>(f32, layer, quant)
                               : fwd_of<32, 3, false>(f32, layer, quant);
        case 64: return fwd_of<64, 3, false>(f32, layer, quant);
        case 128: return fwd_of<128, 3, false>(f32, layer, quant);
    }
    return s.j8 == 2 ? fwd_of<256, 2, false>(f32, layer, quant) : fwd_of<256, 3, false>(f32, layer, quant);
}
template <int THREADS, int TPR, int J8, bool WIDE>
BwdKernel bwd_of(bool f32, bool layer) {
    if (f32)
        return layer ? norm_gate_bwd_kernel<THREADS, TPR, 2 * J8, 4, true, WIDE>
                     : norm_gate_bwd_kernel<THREADS, TPR, 2 * J8, 4, false, WIDE>;
    return layer ? norm_gate_bwd_kernel<THREADS, TPR, J8, 8, true, WIDE> : norm_gate_bwd_kernel<THREADS, TPR, J8, 8, false, WIDE>;
}
BwdKernel backward_kernel(const Split& s, bool f32, bool layer) {
    if (s.ctas > 1) return bwd_of<256, 256, 3, true>(f32, layer);
    switch (s.tpr) {
        case 32: return s.j8 == 1 ? bwd_of<384, 32, 1, false>(f32, layer) : bwd_of<384, 32, 2, false>(f32, layer);
        case 64: return bwd_of<384, 64, 2, false>(f32, layer);
        case 96: return bwd_of<384, 96, 2, false>(f32, layer);
        case 128: return bwd_of<384, 128, 2, false>(f32, layer);
        case 192: return bwd_of<384, 192, 2, false>(f32, layer);
    }
    return s.j8 == 2 ? bwd_of<256, 256, 2, false>(f32, layer) : bwd_of<256, 256, 3, false>(f32, layer);
}

}  // namespace

int launch_norm_gate(const NormArgs& a0, bool f32, cudaStream_t stream) {
    NormArgs a = a0;
    const Split s = forward_split(a.C);
    const FwdKernel kernel = forward_kernel(s, f32, a.layer, a.codes != nullptr);
    a.cols = s.cols;
    a.slot_bytes = (uint32_t)s.cols * ((f32 ? 4 : 2) + (a.h ? 2 : 0));
    Shape sh;
    const int st = shape_of(reinterpret_cast<const void*>(kernel), s, (size_t)12 * s.cols, a.slot_bytes, a.rows, sh);
    if (st != FP4ATTN_OK) return st;
    a.slots = sh.slots;
    return launch(kernel, a, s, sh, stream);
}

// Parts of a sample's rows: the longest way of a team, ceil(groups * parts /
// clusters) items of its share of ceil(rows / parts) rows each, is what the
// launch takes.
int64_t norm_backward_parts(int64_t rows, int64_t C, int64_t groups) {
    if (rows == 0 || groups == 0) return 1;
    const Split s = backward_split(C);
    const int64_t rpg = rows / groups, clusters = 148 / s.ctas;
    if (s.ctas > 1) {
        // how many clusters run at once is not known here: short items even that out
        const int64_t many = (4 * clusters + groups - 1) / groups;
        return many < rpg ? many : rpg;
    }
    // the most parts for each number of rounds: more of them are shorter
    int64_t best = 1, cost = -1;
    for (int64_t rounds = 1; rounds <= 4; ++rounds) {
        int64_t p = rounds * clusters / groups;
        p = p < 1 ? 1 : p > rpg ? rpg : p;
        const int64_t part = (rpg + p - 1) / p;
        const int64_t c = ((groups * p + clusters - 1) / clusters) * ((part + s.teams - 1) / s.teams);
        if (cost < 0 || c < cost) {
            cost = c;
            best = p;
        }
    }
    return best;
}

int launch_norm_gate_backward(const NormBwdArgs& a0, bool f32, cudaStream_t stream) {
    NormBwdArgs a = a0;
    const Split s = backward_split(a.C);
    const BwdKernel kernel = backward_kernel(s, f32, a.layer);
    a.cols = s.cols;
    a.slot_bytes = (uint32_t)s.cols * ((f32 ? 4 : 2) * (a.dy ? 2 : 1) + (a.h ? 4 : 2));
    Shape sh;
    const int st = shape_of(reinterpret_cast<const void*>(kernel), s, (size_t)(s.teams > 1 ? 20 : 8) * s.cols, a.slot_bytes,
                            a.groups * a.parts, sh);
    if (st != FP4ATTN_OK) return st;
    a.slots = sh.slots;
    if (launch(kernel, a, s, sh, stream) != FP4ATTN_OK) return FP4ATTN_ERR_CUDA;
    const int64_t blocks = (a.C + 31) / 32;
    if (launch_behind(norm_join_kernel, dim3((unsigned)(blocks * a.groups)), 256, 0, stream, 1, a) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    if (a.groups > 1 && (a.dpre || a.dpost) &&
        launch_behind(norm_weights_kernel, dim3((unsigned)blocks), 256, 0, stream, 1, a) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    return FP4ATTN_OK;
}

}  // namespace fp4attn
