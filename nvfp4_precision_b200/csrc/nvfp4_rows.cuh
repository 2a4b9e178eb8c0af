// NVFP4 rows for the linear layers: the quantiser of one 16-value block and
// the tile layout of the block scales, shared by the row quantiser and the
// gated norm.
#pragma once
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace fp4attn {

// Launch that may start before the kernel in front of it has finished (see
// pdl_wait): hides most of a launch's latency in chains of short kernels.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                                 unsigned cluster, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Scales of a matrix of `rows` x K values lie in tiles of 128 rows x 64
// channels (four blocks), 512 bytes each, tiles of one row block in channel
// order: the word of row r and 64-channel chunk c (its four scales) is word
// 4 (r % 32) + (r % 128) / 32 of tile (r / 128) * chunks + c.  That is the
// form in which tcgen05.cp takes scale factors, so the product copies tiles
// from memory to TMEM without touching them; chunks = ceil(K / 64), and the
// scales of channels past K are 0.
__host__ __device__ inline int64_t scale_chunks(int64_t K) { return (K + 63) / 64; }
__host__ __device__ inline int64_t scale_tile_bytes(int64_t rows, int64_t K) {
    return (rows + 127) / 128 * scale_chunks(K) * 512;
}
__device__ __forceinline__ uint32_t scale_word_in_tile(uint32_t row_in_block) {
    return 4u * (row_in_block & 31u) + (row_in_block >> 5);
}

// max(a, b) that keeps a NaN of either
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Largest magnitudes of a unit of bf16 values, a pair in a word, NaN kept.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
__device__ __forceinline__ uint32_t abs_pair(uint32_t a) { return a & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t amax_pair(uint2 w) { return max_pair(abs_pair(w.x), abs_pair(w.y)); }
__device__ __forceinline__ uint32_t amax_pair(uint4 w) {
    return max_pair(amax_pair(make_uint2(w.x, w.y)), amax_pair(make_uint2(w.z, w.w)));
}

// Scale byte and reciprocal of one block with largest magnitude a:
// s = E4M3(fl(fl(a / 6) / g)), inv = fl(1 / fl(g s)), 0 when s is 0.  The same
// steps as the Q and K prologue's, so equal rows get equal bytes from both.
__device__ __forceinline__ void row_block_scale(float a, float g, uint32_t& s, float& inv) {
    float t = div6_rn(a);
    if (g != 1.0f) t = __fdiv_rn(t, g);
    s = cvt_e4m3(t) & 0x7Fu;
    const float sd = ue4m3_value(s);
    inv = (sd != 0.0f) ? __frcp_rn(__fmul_rn(g, sd)) : 0.0f;
}

// The same for many blocks under one g, from two small tables: the scale of a
// block is a non-decreasing function F of its largest magnitude a, so a guess
// within one step (a times 1 / (6 g), rounded to E4M3) is put right by
// comparing a with the smallest values that reach the guess and the step above
// it.  No divide, and the same bits: the table is made with the definition.
//   least[c]  smallest a whose scale byte is at least c (c = 1..126); 0 and
//             infinity at the ends
//   recip[c]  fl(1 / fl(g s)), 0 for c = 0
struct ScaleTable {
    float least[129];
    float recip[128];
    float guess;  // 1 / (6 g); 0: g is out of the range where the guess holds
};

// Made by the first 128 threads of a block; the caller synchronises behind it.
__device__ __forceinline__ void make_scale_table(ScaleTable& tab, float g, int t) {
    if (t >= 128) return;
    // beyond these, fl(a / 6) or the guess could be subnormal or overflow where the scale is neither 0 nor 448
    const bool usable = g > 7.888609052210118e-31f && g < 1.2676506002282294e30f;  // 2^-100, 2^100
    const float sd = ue4m3_value((uint32_t)t);
    tab.recip[t] = t ? __frcp_rn(__fmul_rn(g, sd)) : 0.0f;
    if (t == 0) tab.guess = usable ? __frcp_rn(6.0f * g) : 0.0f;
    if (t == 0) tab.least[0] = 0.0f;
    if (t == 127) tab.least[127] = tab.least[128] = INFINITY;
    if (t == 0 || t == 127 || !usable) return;
    auto reaches = [&](float a) {
        float q = div6_rn(a);
        if (g != 1.0f) q = __fdiv_rn(q, g);
        return (cvt_e4m3(q) & 0x7Fu) >= (uint32_t)t;
    };
    // start at the border between the two scales and walk to the exact value (a
    // few units in the last place; bounded in any case)
    float a = 6.0f * g * (0.5f * (sd + ue4m3_value((uint32_t)t - 1)));
    for (int i = 0; i < 16 && !reaches(a); ++i) a = __int_as_float(__float_as_int(a) + 1);
    for (int i = 0; i < 16 && reaches(__int_as_float(__float_as_int(a) - 1)); ++i) a = __int_as_float(__float_as_int(a) - 1);
    tab.least[t] = a;
}

__device__ __forceinline__ void row_block_scale(const ScaleTable& tab, float guess, float a, float g, uint32_t& s,
                                                float& inv) {
    if (guess != 0.0f) {
        uint32_t c = cvt_e4m3(a * guess) & 0x7Fu;
        c = c > 126u ? 126u : c;
        const float lo = tab.least[c], hi = tab.least[c + 1];
        c = a < lo ? c - 1u : c;
        c = a >= hi ? c + 1u : c;
        c = c > 126u ? 126u : c;  // an infinite a
        s = c;
        inv = tab.recip[c];
    } else {
        row_block_scale(a, g, s, inv);
    }
}

// Smallest computed per-tensor scale and the value it covers.
constexpr float kMinGscale = 5.421010862427522e-20f;  // 2^-64
__device__ __forceinline__ float computed_gscale(float amax) {
    // a NaN amax stays one (and is reported); fmaxf would drop it
    const float g = __fdiv_rn(amax, 2688.0f);  // 6 * 448
    return g < kMinGscale ? kMinGscale : g;
}

__device__ __forceinline__ bool bad_gscale(float g) { return !(g > 0.0f && g < INFINITY); }

__device__ __forceinline__ void raise_status(int* status, int code) {
    if (status) atomicCAS(status, 0, code);
}

}  // namespace fp4attn
