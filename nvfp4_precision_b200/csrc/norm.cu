// The norms around a branch, forward: see norm_teams.cuh for what both directions
// share.
#include "norm_teams.cuh"

namespace fp4attn {

namespace {

// ------------------------------------------------------------- forward --
//
// The products of the vectors (A = gate post_weight, B = pre_weight
// (1 + scale), S = shift) stand in shared memory, shared by the CTA's teams,
// which take turns down the rows of one sample after another; that leaves
// registers for 512 threads, twice the warps of the backward to hide the
// reductions and the quantiser behind.

// FULL: the row fills its team, no thread is left without channels.  The quantised
// forms have it (without quantisation the same within 2%), for teams of 128 and 256
// threads.  Without and with it, layer norm of bf16 and fp32 rows, RMS norm of both:
//   36864 x 6144   373 -> 344, 485 -> 476, 307 -> 295, 440 -> 406 us
//   55296 x 4096   412 -> 373, 535 -> 522, 336 -> 322, 477 -> 453
// Narrower teams have no such instances: bf16 rows would gain 10 to 16% (147456 x
// 1536: 330 -> 289 us), fp32 RMS norms lose at some widths (294912 x 768: 403 -> 434).
template <int TPR, int J, int U, bool LAYER, bool QUANT, bool WIDE, bool FULL>
__global__ void __launch_bounds__(FWD_THREADS, 1) norm_gate_kernel(const __grid_constant__ NormArgs a) {
    constexpr int TEAMS = FWD_THREADS / TPR, ES = U == 4 ? 4 : 2, P = U / 2;
    using TeamT = Team<TPR, 2, WIDE>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[TEAMS * MAX_SLOTS];
    __shared__ __align__(16) float scratch[TEAMS * TeamT::SCRATCH];
    __shared__ uint64_t team_bars[2 * TEAMS];
    __shared__ int abort_all;
    __shared__ ScaleTable table;  // not used (and not there) unless QUANT
    const int t = threadIdx.x % TPR;
    TeamT team;
    team.index = threadIdx.x / TPR;
    team.scratch = scratch + team.index * TeamT::SCRATCH;
    team.phase = 0;
    team.rank = WIDE ? cluster_ctarank() : 0;
    team.ranks = WIDE ? cluster_nctarank() : 1;
    team.bars = smem_u32(&team_bars[2 * team.index]);
    team.turn = 0;
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
    if (WIDE && threadIdx.x < 2 * TEAMS) mbar_init(smem_u32(&team_bars[threadIdx.x]), team.ranks * TeamT::warps);
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
                if ((FULL || u < NU)) {
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
                            if (all || (FULL || t + TPR * j < NU))
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
                    if ((FULL || t + TPR * j < NU)) {
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
                    if ((FULL || u < NU) && FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status)) store_res(y_at, u, y[j]);
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
                        if (all || (FULL || t + TPR * j < NU))
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
                if ((FULL || u < NU)) {
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
                const bool on = (FULL || u < NU) && FP4ATTN_IN_BOUNDS(row < a.rows && c0 + U * u + U <= a.C, a.status);
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

using FwdKernel = void (*)(const NormArgs);

template <int TPR, int J8, bool WIDE, bool FULL = false>
FwdKernel quant_of(bool f32, bool layer) {
    if (f32)
        return layer ? norm_gate_kernel<TPR, 2 * J8, 4, true, true, WIDE, FULL> : norm_gate_kernel<TPR, 2 * J8, 4, false, true, WIDE, FULL>;
    return layer ? norm_gate_kernel<TPR, J8, 8, true, true, WIDE, FULL> : norm_gate_kernel<TPR, J8, 8, false, true, WIDE, FULL>;
}
template <int TPR, int J8, bool WIDE>
FwdKernel fwd_of(bool f32, bool layer, bool quant) {
    if (quant) return quant_of<TPR, J8, WIDE>(f32, layer);
    if (f32)
        return layer ? norm_gate_kernel<TPR, 2 * J8, 4, true, false, WIDE, false> : norm_gate_kernel<TPR, 2 * J8, 4, false, false, WIDE, false>;
    return layer ? norm_gate_kernel<TPR, J8, 8, true, false, WIDE, false> : norm_gate_kernel<TPR, J8, 8, false, false, WIDE, false>;
}
FwdKernel forward_kernel(const Split& s, bool f32, bool layer, bool quant) {
    if (s.ctas > 1) return fwd_of<256, 3, true>(f32, layer, quant);
    if (quant && s.tpr >= 128 && s.cols == 8 * s.tpr * s.j8) {
        if (s.tpr == 128) return quant_of<128, 3, false, true>(f32, layer);
        return s.j8 == 2 ? quant_of<256, 2, false, true>(f32, layer) : quant_of<256, 3, false, true>(f32, layer);
    }
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

}  // namespace fp4attn
