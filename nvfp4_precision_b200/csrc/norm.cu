// The two norms around a block's branch, with its gate, its residual and the
// modulation of the next one, and their gradients:
//
//   y = x + gate * (post_weight * norm(h))
//   z = norm(y) * pre_weight * (1 + scale) + shift
//   norm(v) = v / sqrt(mean(v^2) + eps), or the same of v - mean(v)
//
// (DiT blocks: Peebles and Xie, "Scalable Diffusion Models with Transformers",
// 2023; a norm on the branch's output as well: Ding et al., "CogView", 2021.)
// Both directions are bound by HBM: every row is read once and written once,
// so what matters is that enough bytes are on their way at any time.
//   * A team of threads holds one row in registers (statistics are sums over
//     the team, fp32, in a fixed order) and walks down a contiguous range of
//     rows.
//   * The rows ahead come in by bulk copies into a ring in shared memory, one
//     ring per team; a slot is filled again as soon as its row is in registers,
//     so loads stay in flight through the reductions and the stores.
//   * The per-channel vectors are read by every row and stay in L1.
// The forward's z can leave as NVFP4 rows (rounded to bf16 first, as the
// quantiser of a bf16 z would see it), so that the next linear layer reads
// 9/16 byte a value instead of writing, reading and quantising 2-byte ones.
// The backward's sums down the columns stay in registers over a team's rows;
// the teams' parts meet in the workspace and are added in order: no atomics,
// equal calls give equal bits.
#include <cuda_bf16.h>

#include "nvfp4_rows.cuh"

namespace fp4attn {

namespace {

constexpr int NTHREADS = 512;
constexpr uint64_t kLimitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait
constexpr int MAX_SLOTS = 4;

template <int TPR>
__device__ __forceinline__ void team_sync(int team) {
    if constexpr (TPR == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TPR) : "memory");
}

// Sums over the team of K values per thread, the same bits in every thread.
// `scratch` holds two buffers that alternate, so one barrier per sum is enough.
template <int TPR, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float* scratch, int& phase, int team) {
    constexpr int W = TPR / 32;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (W == 1) {
        __syncwarp();
    } else {
        float* at = scratch + phase * (4 * W);
        phase ^= 1;
        const int warp = (threadIdx.x % TPR) >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) at[k * W + warp] = v[k];
        team_sync<TPR>(team);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += at[k * W + w];
            v[k] = s;
        }
    }
}

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(x[i]);
        v[2 * i + 1] = bf16hi(x[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void unpack4(uint2 w, float (&v)[4]) {
    v[0] = bf16lo(w.x);
    v[1] = bf16hi(w.x);
    v[2] = bf16lo(w.y);
    v[3] = bf16hi(w.y);
}
__device__ __forceinline__ uint4 ldg16(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 ones
__device__ __forceinline__ uint4 ldg16_or(const __nv_bfloat16* p, int64_t at, uint32_t w) {
    return p ? ldg16(p + at) : make_uint4(w, w, w, w);
}
__device__ __forceinline__ uint2 ldg8_or(const __nv_bfloat16* p, int64_t at, uint32_t w) {
    return p ? ldg8(p + at) : make_uint2(w, w);
}

// One team's ring: `slots` rows on their way or in use.  Thread 0 of the team
// fills a slot once every thread has its row in registers.
struct Ring {
    uint8_t* buf;
    uint32_t bars;   // shared address of the slots' barriers
    uint32_t slot_bytes;
    int slots;
};

// ------------------------------------------------------------- forward --

template <int TPR, int J, bool F32, bool QUANT>
__global__ void __launch_bounds__(NTHREADS) norm_gate_kernel(const __grid_constant__ NormArgs a) {
    constexpr int TEAMS = NTHREADS / TPR, ES = F32 ? 4 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[TEAMS * MAX_SLOTS];
    __shared__ __align__(16) float scratch_all[TEAMS * 8 * (TPR / 32)];
    __shared__ int abort_all;
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int C = a.C, NV = C / 8;
    float* scratch = scratch_all + team * 8 * (TPR / 32);
    if (threadIdx.x == 0) abort_all = 0;
    if (threadIdx.x < TEAMS * MAX_SLOTS) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
    fence_mbar_init();
    __syncthreads();
    if (a.pdl) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    volatile int* abort_flag = &abort_all;

    const bool has_h = a.h != nullptr;
    const uint32_t x_bytes = (uint32_t)C * ES, h_bytes = has_h ? (uint32_t)C * 2 : 0;
    uint8_t* ring = smem + (size_t)team * a.slots * a.slot_bytes;
    const uint32_t ring_u = smem_u32(ring);
    const int64_t team_id = blockIdx.x + (int64_t)gridDim.x * team, n_teams = (int64_t)gridDim.x * TEAMS;
    const int64_t r0 = a.rows * team_id / n_teams, r1 = a.rows * (team_id + 1) / n_teams;
    auto fill = [&](int64_t row, int slot) {
        const uint32_t bar = smem_u32(&bars[team * MAX_SLOTS + slot]);
        const uint32_t at = ring_u + a.slot_bytes * slot;
        mbar_arrive_expect_tx(bar, x_bytes + h_bytes);
        bulk_load(at, static_cast<const uint8_t*>(a.x) + row * a.ldx * ES, x_bytes, bar);
        if (has_h) bulk_load(at + x_bytes, a.h + row * a.ldh, h_bytes, bar);
    };
    int64_t next = r0;
    if (t == 0)
        for (int s = 0; s < a.slots && next < r1; ++s, ++next) fill(next, s);
    const float gz = QUANT ? (a.gz ? __ldg(a.gz) : 1.0f) : 1.0f;
    if (QUANT && blockIdx.x == 0 && threadIdx.x == 0 && bad_gscale(gz)) raise_status(a.status, FP4ATTN_ERR_RANGE);
    const float inv_c = 1.0f / (float)C;
    bool finite = true;
    int phase = 0, slot = 0;
    uint32_t parity = 0;
    int64_t group = r0 < r1 ? r0 / a.rows_per_group : 0;
    int64_t group_end = (group + 1) * a.rows_per_group;
    for (int64_t row = r0; row < r1; ++row) {
        if (row >= group_end) {
            ++group;
            group_end += a.rows_per_group;
        }
        const bool ok = mbar_wait(smem_u32(&bars[team * MAX_SLOTS + slot]), parity, abort_flag, a.status, kLimitNs);
        const uint8_t* at = ring + (size_t)a.slot_bytes * slot;
        float yv[J][8];
        uint4 hv[J], pv[J], gv[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int v = t + TPR * j;
            if (v < NV) {
                if constexpr (F32) {
                    const float4 lo = reinterpret_cast<const float4*>(at)[2 * v];
                    const float4 hi = reinterpret_cast<const float4*>(at)[2 * v + 1];
                    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) yv[j][i] = f[i];
                } else {
                    unpack8(reinterpret_cast<const uint4*>(at)[v], yv[j]);
                }
                if (has_h) {
                    hv[j] = reinterpret_cast<const uint4*>(at + x_bytes)[v];
                    pv[j] = ldg16_or(a.post, 8 * v, kOnes);
                    gv[j] = ldg16_or(a.gate, group * a.lgate + 8 * v, kOnes);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) yv[j][i] = 0.0f;
                hv[j] = pv[j] = gv[j] = make_uint4(0, 0, 0, 0);
            }
            // a row that never came (its wait ran out) must not pass for one
            if (!ok)
#pragma unroll
                for (int i = 0; i < 8; ++i) yv[j][i] = __int_as_float(0x7FC00000);
        }
        if (!has_h) team_sync<TPR>(team);
        if (has_h) {
            float mean = 0.0f, q[1] = {0.0f};
            if (a.layer) {
                float s[1] = {0.0f};
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float f[8];
                    unpack8(hv[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[0] += f[i];
                }
                team_sum<TPR, 1>(s, scratch, phase, team);
                mean = s[0] * inv_c;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[8];
                unpack8(hv[j], f);
                if (t + TPR * j < NV)
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[0] = __fmaf_rn(f[i] - mean, f[i] - mean, q[0]);
            }
            team_sum<TPR, 1>(q, scratch, phase, team);
            const float r = rsqrtf(__fmaf_rn(q[0], inv_c, a.eps));
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[8], p[8], g[8];
                unpack8(hv[j], f);
                unpack8(pv[j], p);
                unpack8(gv[j], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) yv[j][i] = __fmaf_rn(g[i] * p[i], (f[i] - mean) * r, yv[j][i]);
            }
        }
        // every thread has passed a barrier behind its loads: the slot is free
        if (t == 0 && next < r1 && !*abort_flag) fill(next++, slot);
        if (++slot == a.slots) {
            slot = 0;
            parity ^= 1;
        }
        if (a.y) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int v = t + TPR * j;
                if (v < NV && FP4ATTN_IN_BOUNDS(row < a.rows && 8 * v + 8 <= C, a.status)) {
                    if constexpr (F32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.y) + row * a.ldy + 8 * v);
                        dst[0] = make_float4(yv[j][0], yv[j][1], yv[j][2], yv[j][3]);
                        dst[1] = make_float4(yv[j][4], yv[j][5], yv[j][6], yv[j][7]);
                    } else {
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * a.ldy + 8 * v) = pack8(yv[j]);
                    }
                }
            }
        }
        if (!QUANT && !a.z) continue;
        uint4 sc[J], sh[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int v = t + TPR * j;
            pv[j] = sc[j] = sh[j] = make_uint4(0, 0, 0, 0);
            if (v < NV) {
                pv[j] = ldg16_or(a.pre, 8 * v, kOnes);
                sc[j] = ldg16_or(a.scale, group * a.lscale + 8 * v, 0u);
                sh[j] = ldg16_or(a.shift, group * a.lshift + 8 * v, 0u);
            }
        }
        float mean = 0.0f, q[1] = {0.0f};
        if (a.layer) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (t + TPR * j < NV)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[0] += yv[j][i];
            team_sum<TPR, 1>(s, scratch, phase, team);
            mean = s[0] * inv_c;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (t + TPR * j < NV)
#pragma unroll
                for (int i = 0; i < 8; ++i) q[0] = __fmaf_rn(yv[j][i] - mean, yv[j][i] - mean, q[0]);
        team_sum<TPR, 1>(q, scratch, phase, team);
        const float r = rsqrtf(__fmaf_rn(q[0], inv_c, a.eps));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int v = t + TPR * j;
            float p[8], s[8], b[8], z[8];
            unpack8(pv[j], p);
            unpack8(sc[j], s);
            unpack8(sh[j], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = __fmaf_rn((yv[j][i] - mean) * r, __fmaf_rn(p[i], s[i], p[i]), b[i]);
            const uint4 w = pack8(z);
            if constexpr (!QUANT) {
                if (v < NV && FP4ATTN_IN_BOUNDS(row < a.rows && 8 * v + 8 <= C, a.status))
                    *reinterpret_cast<uint4*>(a.z + row * a.ldz + 8 * v) = w;
            } else {
                // two lanes share a block of 16 values, eight a word of four scales
                unpack8(w, z);
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(z[i]));
                if (v >= NV) m = 0.0f;
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
                finite = finite && (m < INFINITY);
                uint32_t s8;
                float inv;
                row_block_scale(m, gz, s8, inv);
                if (v < NV && FP4ATTN_IN_BOUNDS(row < a.rows && 8 * v + 8 <= C, a.status))
                    *reinterpret_cast<uint32_t*>(a.codes + row * (C / 2) + 4 * v) = row_codes8(z, inv);
                uint32_t word = s8 << (8 * ((v >> 1) & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
                const int64_t off = ((row >> 7) * a.chunks + (v >> 3)) * 128 + scale_word_in_tile((uint32_t)row & 127);
                if ((v & 7) == 0 && v < NV && FP4ATTN_IN_BOUNDS(4 * off + 4 <= scale_tile_bytes(a.rows, C), a.status))
                    reinterpret_cast<uint32_t*>(a.scales)[off] = word;
            }
        }
    }
    if (QUANT && !finite) raise_status(a.status, FP4ATTN_ERR_RANGE);
    if (t == 0 && *abort_flag) {
        // this team's own copies land before it leaves (bounded)
        int dummy = 0;
        for (int s = 0; s < a.slots; ++s)
            for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(smem_u32(&bars[team * MAX_SLOTS + s]), ph, &dummy, nullptr, 200000000ull);
    }
}

// ------------------------------------------------------------ backward --
//
// With n = norm(y) = r (y - mean), dn = dz pre (1 + scale):
//   dx = dy + r (dn - n mean(dn n) - [layer] mean(dn))
// and with m = norm(h), dm = dx gate post:
//   dh = r_h (dm - m mean(dm m) - [layer] mean(dm))
// Sums down the rows of a sample: dz, dz n, dx m.

template <int TPR, int J, bool F32>
__global__ void __launch_bounds__(NTHREADS) norm_gate_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
    constexpr int TEAMS = NTHREADS / TPR, ES = F32 ? 4 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[TEAMS * MAX_SLOTS];
    __shared__ __align__(16) float scratch_all[TEAMS * 8 * (TPR / 32)];
    __shared__ int abort_all;
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int C = a.C, NV = C / 4;
    float* scratch = scratch_all + team * 8 * (TPR / 32);
    if (threadIdx.x == 0) abort_all = 0;
    if (threadIdx.x < TEAMS * MAX_SLOTS) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
    fence_mbar_init();
    __syncthreads();
    volatile int* abort_flag = &abort_all;

    const bool has_h = a.h != nullptr, has_dy = a.dy != nullptr;
    const uint32_t res_bytes = (uint32_t)C * ES, half_bytes = (uint32_t)C * 2;
    // a slot: y, dy (residual type), dz, h (bf16)
    const uint32_t at_dy = res_bytes, at_dz = at_dy + (has_dy ? res_bytes : 0), at_h = at_dz + half_bytes;
    const uint32_t row_bytes = at_h + (has_h ? half_bytes : 0);
    uint8_t* ring = smem + (size_t)team * a.slots * a.slot_bytes;
    const uint32_t ring_u = smem_u32(ring);
    const int64_t team_id = blockIdx.x + (int64_t)gridDim.x * team, n_teams = (int64_t)gridDim.x * TEAMS;
    const int64_t items = a.groups * a.parts;
    auto item_begin = [&](int64_t item, int64_t& begin, int64_t& end) {
        const int64_t g = item / a.parts, p = item - g * a.parts;
        begin = g * a.rows_per_group + a.rows_per_group * p / a.parts;
        end = g * a.rows_per_group + a.rows_per_group * (p + 1) / a.parts;
    };
    // the rows ahead, over the items of this team
    int64_t ahead_item = team_id, ahead = 0, ahead_end = 0;
    if (ahead_item < items) item_begin(ahead_item, ahead, ahead_end);
    auto fill_next = [&](int slot) {
        while (ahead >= ahead_end) {
            ahead_item += n_teams;
            if (ahead_item >= items) {
                ahead_item = items;
                return;
            }
            item_begin(ahead_item, ahead, ahead_end);
        }
        const int64_t row = ahead++;
        const uint32_t bar = smem_u32(&bars[team * MAX_SLOTS + slot]);
        const uint32_t at = ring_u + a.slot_bytes * slot;
        mbar_arrive_expect_tx(bar, row_bytes);
        bulk_load(at, static_cast<const uint8_t*>(a.y) + row * a.ldy * ES, res_bytes, bar);
        if (has_dy) bulk_load(at + at_dy, static_cast<const uint8_t*>(a.dy) + row * a.lddy * ES, res_bytes, bar);
        bulk_load(at + at_dz, a.dz + row * a.lddz, half_bytes, bar);
        if (has_h) bulk_load(at + at_h, a.h + row * a.ldh, half_bytes, bar);
    };
    if (t == 0 && ahead_item < items)
        for (int s = 0; s < a.slots && ahead_item < items; ++s) fill_next(s);
    const float inv_c = 1.0f / (float)C;
    int phase = 0, slot = 0;
    uint32_t parity = 0;
    for (int64_t item = team_id; item < items; item += n_teams) {
        int64_t begin, end;
        item_begin(item, begin, end);
        const int64_t group = item / a.parts;
        float s_dz[J][4], s_dzn[J][4], s_dxm[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_dz[j][i] = s_dzn[j][i] = s_dxm[j][i] = 0.0f;
        for (int64_t row = begin; row < end; ++row) {
            const bool ok = mbar_wait(smem_u32(&bars[team * MAX_SLOTS + slot]), parity, abort_flag, a.status, kLimitNs);
            const uint8_t* at = ring + (size_t)a.slot_bytes * slot;
            float y[J][4], dy[J][4];
            uint2 dz[J], h[J];
            // sums of the first pass: y, dn, h (layer norm), then their squares and dn y
            float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int v = t + TPR * j;
                dz[j] = h[j] = make_uint2(0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[j][i] = dy[j][i] = 0.0f;
                if (v < NV) {
                    if constexpr (F32) {
                        const float4 f = reinterpret_cast<const float4*>(at)[v];
                        y[j][0] = f.x, y[j][1] = f.y, y[j][2] = f.z, y[j][3] = f.w;
                        if (has_dy) {
                            const float4 d = reinterpret_cast<const float4*>(at + at_dy)[v];
                            dy[j][0] = d.x, dy[j][1] = d.y, dy[j][2] = d.z, dy[j][3] = d.w;
                        }
                    } else {
                        unpack4(reinterpret_cast<const uint2*>(at)[v], y[j]);
                        if (has_dy) unpack4(reinterpret_cast<const uint2*>(at + at_dy)[v], dy[j]);
                    }
                    dz[j] = reinterpret_cast<const uint2*>(at + at_dz)[v];
                    if (has_h) h[j] = reinterpret_cast<const uint2*>(at + at_h)[v];
                }
                if (!ok)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[j][i] = __int_as_float(0x7FC00000);
            }
            auto dn_of = [&](int j, float (&dn)[4], float (&d)[4]) {
                // dz and dz pre (1 + scale)
                const int v = t + TPR * j;
                uint2 pw = make_uint2(0, 0), sw = make_uint2(0, 0);
                if (v < NV) {
                    pw = ldg8_or(a.pre, 4 * v, kOnes);
                    sw = ldg8_or(a.scale, group * a.lscale + 4 * v, 0u);
                }
                float p[4], s[4];
                unpack4(dz[j], d);
                unpack4(pw, p);
                unpack4(sw, s);
#pragma unroll
                for (int i = 0; i < 4; ++i) dn[i] = d[i] * __fmaf_rn(p[i], s[i], p[i]);
            };
            float mean_y = 0.0f, mean_h = 0.0f, mean_dn = 0.0f;
            if (a.layer) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float dn[4], d[4], hh[4];
                    dn_of(j, dn, d);
                    unpack4(h[j], hh);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s1[0] += y[j][i];
                        s1[1] += dn[i];
                        s1[2] += hh[i];
                    }
                }
                team_sum<TPR, 3>(s1, scratch, phase, team);
                mean_y = s1[0] * inv_c;
                mean_dn = s1[1] * inv_c;
                mean_h = s1[2] * inv_c;
            }
            float s2[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float dn[4], d[4], hh[4];
                dn_of(j, dn, d);
                unpack4(h[j], hh);
                if (t + TPR * j < NV)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[j][i] -= mean_y;
                        s2[0] = __fmaf_rn(y[j][i], y[j][i], s2[0]);
                        s2[1] = __fmaf_rn(dn[i], y[j][i], s2[1]);
                        s2[2] = __fmaf_rn(hh[i] - mean_h, hh[i] - mean_h, s2[2]);
                    }
            }
            team_sum<TPR, 3>(s2, scratch, phase, team);
            if (t == 0 && ahead_item < items && !*abort_flag) fill_next(slot);
            if (++slot == a.slots) {
                slot = 0;
                parity ^= 1;
            }
            const float ry = rsqrtf(__fmaf_rn(s2[0], inv_c, a.eps)), rh = rsqrtf(__fmaf_rn(s2[2], inv_c, a.eps));
            const float c1 = s2[1] * inv_c * ry;  // mean(dn n)
            float s3[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int v = t + TPR * j;
                float dn[4], d[4];
                dn_of(j, dn, d);
                uint2 pw = make_uint2(0, 0), gw = make_uint2(0, 0);
                if (has_h && v < NV) {
                    pw = ldg8_or(a.post, 4 * v, kOnes);
                    gw = ldg8_or(a.gate, group * a.lgate + 4 * v, kOnes);
                }
                float p[4], g[4], hh[4];
                unpack4(pw, p);
                unpack4(gw, g);
                unpack4(h[j], hh);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float n = y[j][i] * ry;
                    s_dz[j][i] += d[i];
                    s_dzn[j][i] = __fmaf_rn(d[i], n, s_dzn[j][i]);
                    const float dx = __fmaf_rn(ry, dn[i] - mean_dn - n * c1, dy[j][i]);
                    const float m = (hh[i] - mean_h) * rh;
                    s_dxm[j][i] = __fmaf_rn(dx, m, s_dxm[j][i]);
                    const float dm = dx * (g[i] * p[i]);
                    s3[0] = __fmaf_rn(dm, m, s3[0]);
                    s3[1] += dm;
                    dy[j][i] = dx;
                    y[j][i] = dm;
                }
                if (v < NV && FP4ATTN_IN_BOUNDS(row < a.rows && 4 * v + 4 <= C, a.status)) {
                    if constexpr (F32)
                        *reinterpret_cast<float4*>(static_cast<float*>(a.dx) + row * a.lddx + 4 * v) =
                            make_float4(dy[j][0], dy[j][1], dy[j][2], dy[j][3]);
                    else
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dx) + row * a.lddx + 4 * v) =
                            make_uint2(pack_bf16x2(dy[j][0], dy[j][1]), pack_bf16x2(dy[j][2], dy[j][3]));
                }
            }
            if (!has_h) continue;
            team_sum<TPR, 2>(s3, scratch, phase, team);
            const float c2 = s3[0] * inv_c, mean_dm = a.layer ? s3[1] * inv_c : 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int v = t + TPR * j;
                float hh[4], o[4];
                unpack4(h[j], hh);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = (hh[i] - mean_h) * rh;
                    o[i] = rh * (y[j][i] - mean_dm - m * c2);
                }
                if (v < NV && FP4ATTN_IN_BOUNDS(row < a.rows && 4 * v + 4 <= C, a.status))
                    *reinterpret_cast<uint2*>(a.dh + row * a.lddh + 4 * v) =
                        make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            }
        }
        float* part = a.part + item * 3 * (int64_t)C;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int v = t + TPR * j;
            if (v < NV && FP4ATTN_IN_BOUNDS(item < items, a.status)) {
                reinterpret_cast<float4*>(part)[v] = make_float4(s_dz[j][0], s_dz[j][1], s_dz[j][2], s_dz[j][3]);
                reinterpret_cast<float4*>(part + C)[v] = make_float4(s_dzn[j][0], s_dzn[j][1], s_dzn[j][2], s_dzn[j][3]);
                reinterpret_cast<float4*>(part + 2 * C)[v] =
                    make_float4(s_dxm[j][0], s_dxm[j][1], s_dxm[j][2], s_dxm[j][3]);
            }
        }
    }
    if (t == 0 && *abort_flag) {
        int dummy = 0;
        for (int s = 0; s < a.slots; ++s)
            for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(smem_u32(&bars[team * MAX_SLOTS + s]), ph, &dummy, nullptr, 200000000ull);
    }
}

// Adds a sample's parts in order (32 columns by 8 shares of the parts per CTA;
// the shares meet in order) and makes the gradients of its vectors.  With one
// sample the weights' gradients follow at once; with more the sums are kept,
// in the first part's place, for norm_weights_kernel.
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormBwdArgs a) {
    __shared__ float sum[3][8][32];
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

constexpr size_t RING_BYTES = 160 * 1024;  // shared memory of the rings; the rest of the 228 KB serves as L1 for the vectors
constexpr size_t RING_MOST = 200 * 1024;

// Slots per team: as many as fit RING_BYTES, at most MAX_SLOTS; two where
// RING_MOST holds them, else one.
int ring_slots(size_t row_bytes, int teams) {
    int s = (int)(RING_BYTES / (row_bytes * teams));
    if (s > MAX_SLOTS) s = MAX_SLOTS;
    if (s < 2) s = row_bytes * teams * 2 <= RING_MOST ? 2 : 1;
    return s;
}

int sm_count(int& sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    return FP4ATTN_OK;
}

template <int TPR, int J, bool F32, bool QUANT>
int launch_fwd(NormArgs a, cudaStream_t stream) {
    constexpr int TEAMS = NTHREADS / TPR;
    int sms = 0;
    if (sm_count(sms) != FP4ATTN_OK) return FP4ATTN_ERR_CUDA;
    const size_t row = (size_t)a.C * ((F32 ? 4 : 2) + (a.h ? 2 : 0));
    a.slot_bytes = (uint32_t)row;
    a.slots = ring_slots(row, TEAMS);
    const size_t smem = row * TEAMS * a.slots;
    auto kernel = norm_gate_kernel<TPR, J, F32, QUANT>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    const int64_t grid = a.rows < sms ? a.rows : sms;
    kernel<<<(unsigned)grid, NTHREADS, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? FP4ATTN_OK : FP4ATTN_ERR_CUDA;
}

template <int TPR, int J>
int launch_fwd_types(const NormArgs& a, bool f32, cudaStream_t stream) {
    if (a.codes) return f32 ? launch_fwd<TPR, J, true, true>(a, stream) : launch_fwd<TPR, J, false, true>(a, stream);
    return f32 ? launch_fwd<TPR, J, true, false>(a, stream) : launch_fwd<TPR, J, false, false>(a, stream);
}

template <int TPR, int J>
int launch_bwd(NormBwdArgs a, bool f32, cudaStream_t stream) {
    constexpr int TEAMS = NTHREADS / TPR;
    int sms = 0;
    if (sm_count(sms) != FP4ATTN_OK) return FP4ATTN_ERR_CUDA;
    const size_t res = (size_t)a.C * (f32 ? 4 : 2);
    const size_t row = res * (a.dy ? 2 : 1) + (size_t)a.C * (a.h ? 4 : 2);
    a.slot_bytes = (uint32_t)row;
    a.slots = ring_slots(row, TEAMS);
    const size_t smem = row * TEAMS * a.slots;
    auto kernel = f32 ? norm_gate_bwd_kernel<TPR, J, true> : norm_gate_bwd_kernel<TPR, J, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return FP4ATTN_ERR_CUDA;
    const int64_t items = a.groups * a.parts;
    const int64_t grid = items < sms ? items : sms;
    kernel<<<(unsigned)grid, NTHREADS, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FP4ATTN_ERR_CUDA;
    const int64_t blocks = (a.C + 31) / 32;
    norm_join_kernel<<<(unsigned)(blocks * a.groups), 256, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FP4ATTN_ERR_CUDA;
    if (a.groups > 1 && (a.dpre || a.dpost)) {
        norm_weights_kernel<<<(unsigned)blocks, 256, 0, stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return FP4ATTN_ERR_CUDA;
    }
    return FP4ATTN_OK;
}

int bwd_threads_per_row(int64_t C) { return C <= 512 ? 32 : C <= 1024 ? 64 : C <= 2048 ? 128 : C <= 4096 ? 256 : 512; }

}  // namespace

int launch_norm_gate(const NormArgs& a, bool f32, cudaStream_t stream) {
    const int NV = a.C / 8;
    switch ((NV + 31) / 32) {
        case 1: return launch_fwd_types<32, 1>(a, f32, stream);
        case 2: return launch_fwd_types<32, 2>(a, f32, stream);
        case 3: return launch_fwd_types<32, 3>(a, f32, stream);
        case 4: return launch_fwd_types<32, 4>(a, f32, stream);
    }
    if (NV <= 64 * 3) return launch_fwd_types<64, 3>(a, f32, stream);
    if (NV <= 64 * 4) return launch_fwd_types<64, 4>(a, f32, stream);
    if (NV <= 128 * 3) return launch_fwd_types<128, 3>(a, f32, stream);
    if (NV <= 128 * 4) return launch_fwd_types<128, 4>(a, f32, stream);
    if (NV <= 256 * 3) return launch_fwd_types<256, 3>(a, f32, stream);
    if (NV <= 256 * 4) return launch_fwd_types<256, 4>(a, f32, stream);
    if (NV <= 512 * 3) return launch_fwd_types<512, 3>(a, f32, stream);
    return launch_fwd_types<512, 4>(a, f32, stream);
}

// Parts of a sample's rows: the longest work of a team, ceil(groups * parts /
// teams) items of ceil(rows / parts) rows, is what the launch takes.
int64_t norm_backward_parts(int64_t rows, int64_t C, int64_t groups) {
    if (rows == 0 || groups == 0) return 1;
    const int64_t rpg = rows / groups, teams = 148 * (NTHREADS / bwd_threads_per_row(C));
    int64_t most = (4 * teams + groups - 1) / groups;
    if (most > rpg) most = rpg;
    int64_t best = 1, cost = -1;
    for (int64_t p = 1; p <= most; ++p) {
        const int64_t c = ((groups * p + teams - 1) / teams) * ((rpg + p - 1) / p);
        if (cost < 0 || c < cost) {
            cost = c;
            best = p;
        }
    }
    return best;
}

int launch_norm_gate_backward(const NormBwdArgs& a, bool f32, cudaStream_t stream) {
    const int NV = a.C / 4, tpr = bwd_threads_per_row(a.C);
    const int J = (NV + tpr - 1) / tpr;
    switch (tpr) {
        case 32:
            if (J == 1) return launch_bwd<32, 1>(a, f32, stream);
            if (J == 2) return launch_bwd<32, 2>(a, f32, stream);
            return launch_bwd<32, 4>(a, f32, stream);
        case 64: return J == 3 ? launch_bwd<64, 3>(a, f32, stream) : launch_bwd<64, 4>(a, f32, stream);
        case 128: return J == 3 ? launch_bwd<128, 3>(a, f32, stream) : launch_bwd<128, 4>(a, f32, stream);
        case 256: return J == 3 ? launch_bwd<256, 3>(a, f32, stream) : launch_bwd<256, 4>(a, f32, stream);
    }
    if (J == 3) return launch_bwd<512, 3>(a, f32, stream);
    if (J == 4) return launch_bwd<512, 4>(a, f32, stream);
    if (J <= 6) return launch_bwd<512, 6>(a, f32, stream);
    return launch_bwd<512, 8>(a, f32, stream);
}

}  // namespace fp4attn
