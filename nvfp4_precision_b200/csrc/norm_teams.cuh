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
//   * A team of warps holds a row in registers, up to 24 values a thread; the
//     teams of a CTA (one per SM) take turns down a range of rows.  Products of
//     the per-channel vectors (gate post_weight, pre_weight (1 + scale), shift)
//     are made once per range and sample, in shared memory; the backward's sums
//     down the columns stay in registers over the range.  Rows too wide for a CTA
//     are shared by a cluster.
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
// Forward 109568 x 6144, fp32 residual: 1.39 ms, 5.8 TB/s; backward 36864 x 6144:
// bf16 472 us alone (5.8 TB/s; 500 back to back), layer norm 542, fp32 layer norm
// 630 (6.5 TB/s).  The layer norm into NVFP4 is furthest from HBM's rate (36864 x
// 6144: 344 us of 226): half of the issue slots, and the latency of reductions and
// of look-ups that two lanes (four with fp32 rows) make for one block.  Rows shared
// by a cluster run at half (RMS) to a third (layer norm) of narrower rows' rate: 27648
// x 8192 bf16 forward 677 and 885 us, backward 1080 and 1544.
//
// Shared by norm.cu (forward) and norm_bwd.cu: teams, units, the split of a row and
// the launch.
#pragma once
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
// go their own ways, and a row costs no barrier over all of it.  Two barriers take
// turns: a warp that has met the others at its own CTA's barrier knows nothing of
// another CTA's, where arrivals of the same turn may still be under way, so its next
// arrival there must not count for them.  At the turn after that it may: everyone has
// arrived for the one between, and did so behind the first.
template <int TPR, int MAX_K, bool WIDE>
struct Team {
    static constexpr int warps = TPR / 32;
    static constexpr int MAX_WARPS = (warps + 3) / 4 * 4 * (WIDE ? MAX_CLUSTER : 1);
    // floats per team, zeroed: two buffers that alternate
    static constexpr int SCRATCH = warps == 1 && !WIDE ? 4 : 2 * MAX_K * MAX_WARPS;
    float* scratch;
    int index, phase;
    uint32_t rank, ranks;
    // WIDE: this team's two barriers (ranks * warps arrivals), the turns so far, and
    // what a wait needs
    uint32_t bars, turn;
    volatile int* abort_flag;
    int* status;

    // WIDE, behind the lanes' remote stores
    __device__ __forceinline__ void arrive_and_wait() {
        __syncwarp();
        const int lane = threadIdx.x & 31;
        const uint32_t bar = bars + 8u * (turn & 1);
        if (lane < (int)ranks) mbar_arrive_cluster(mapa(bar, (uint32_t)lane));
        mbar_wait_cluster(bar, (turn >> 1) & 1, abort_flag, status, kLimitNs);
        ++turn;
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
// The same pivots for every CTA of a cluster: each CTA's come from the team's own
// first thread.
template <int TPR, int MAX_K, bool WIDE>
__device__ __forceinline__ void share_pivots(Team<TPR, MAX_K, WIDE>& team, float& p, float& q) {
    if constexpr (WIDE) {
        const bool first = threadIdx.x % TPR == 0;
        float v[2] = {first ? p : 0.0f, first ? q : 0.0f};
        team.sum(v);
        p = v[0] / (float)team.ranks;
        q = v[1] / (float)team.ranks;
    }
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
        // the same for every size: another thread may set it between this and the launch
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES) != cudaSuccess)
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

}  // namespace

}  // namespace fp4attn
