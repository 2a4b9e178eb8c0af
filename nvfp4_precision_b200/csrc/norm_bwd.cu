// The norms around a branch, gradients: see norm_teams.cuh for what both directions
// share.
#include "norm_teams.cuh"

namespace fp4attn {

namespace {

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
    __shared__ uint64_t team_bars[2 * TEAMS];
    __shared__ int abort_all;
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
    if (threadIdx.x == 0) abort_all = 0;
    for (int i = threadIdx.x; i < TEAMS * MAX_SLOTS; i += blockDim.x) mbar_init(smem_u32(&bars[i]), 1);
    for (int i = threadIdx.x; i < (int)(sizeof(scratch) / 4); i += blockDim.x) scratch[i] = 0.0f;
    if (WIDE && threadIdx.x < 2 * TEAMS) mbar_init(smem_u32(&team_bars[threadIdx.x]), team.ranks * TeamT::warps);
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
            // of the mean's own.  dx = dy + r dn - r c1 n - r mean(dn); the layer norm
            // adds its three terms first, so that a large dy is rounded once (for the RMS
            // norm's two, added to dy one after the other, that would be one more step)
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
                        const float2 dn = __fmul2_rn(d[i], B[i]);
                        if constexpr (LAYER)
                            g[i] = __fadd2_rn(g[i], __ffma2_rn(dn, ry2, __ffma2_rn(n, c12, md2)));  // dx
                        else
                            g[i] = __ffma2_rn(dn, ry2, __ffma2_rn(n, c12, g[i]));
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

using BwdKernel = void (*)(const NormBwdArgs);

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
