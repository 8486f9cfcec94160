// q4q_attn.cuh -- what the attention kernels share: the layout of the paged 4-bit cache, and the
// row of a head with its norm and rotation.
//
// The cache.  A page holds page_tokens tokens (a power of two, 16 or more) of all key-value heads:
// for each head, for each 16 tokens, one chunk of 18 D bytes (D: head_dim, B = D / 32 blocks):
//   K codes   16 rows of D / 2 bytes, as [4 t][B] words; nibble n of word (t, b): dim 32 b + 8 t + n
//   V codes   2 octets of 4 D bytes, as [8 g][4 p][B] words; the low half of word (g, p, b) is token
//             2p of the octet, the high half token 2p + 1; nibble n of a half: dim 32 b + 4 g + n
//   K scales  [16][B] fp16;  V scales [16][B] fp16
// Values are those of Q4_0 blocks, (code - 8) * d.  A chunk is what a warp of the attention takes at
// a time, in one bulk copy.  The order of the codes is that of the operands of an m16n8k16 MMA: lane
// (g, t) finds the codes of key g in the words that follow one another from t on, of every block the
// same dims, so that an MMA never crosses a block, whose scale is applied to its fp32 sums; and the
// codes of values as pairs of consecutive keys, the depth of the second product.
#pragma once

#include "q4q_mx.cuh"
#include "q4q_mx_tc.cuh"

namespace q4q {

constexpr int KV_GROUP = 16;             // tokens of a chunk

__host__ __device__ constexpr int kv_chunk_bytes(int dim) { return 18 * dim; }
__host__ __device__ __forceinline__ bool kv_dim_ok(int64_t dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 256; }
__host__ __device__ __forceinline__ bool kv_page_ok(int64_t tokens) { return tokens >= KV_GROUP && tokens <= 4096 && (tokens & (tokens - 1)) == 0; }

// Offset of a head's 16 tokens in the cache: pages of 2^page_log tokens.
__device__ __forceinline__ int64_t kv_chunk_offset(int64_t page, int head, int group, int heads, int page_log, int dim) {
    return (((page * heads + head) << (page_log - 4)) + group) * kv_chunk_bytes(dim);
}

// Offsets in a chunk: the K word of token i that holds dims 32 b + 8 t .. + 7, the V half of token i
// that holds dims 32 b + 4 g .. + 3, the scales of token i and block b.
__device__ __forceinline__ int kv_k_word(int i, int t, int b, int dim) { return i * (dim / 2) + (t * (dim / 32) + b) * 4; }
__device__ __forceinline__ int kv_v_half(int i, int g, int b, int dim) {
    return 8 * dim + (i >> 3) * 4 * dim + ((g * 4 + ((i >> 1) & 3)) * (dim / 32) + b) * 4 + (i & 1) * 2;
}
__device__ __forceinline__ int kv_scale(bool v, int i, int b, int dim) { return (v ? 17 : 16) * dim + (i * (dim / 32) + b) * 2; }

// ---------------------------------------------------------- rows of a head --

// A lane holds 8 consecutive values of a row; a row takes LANES lanes (8, 16 or 32, D / 8 of them in
// use), so a warp holds 32 / LANES rows.

// 8 values at p; `align`: of every row's start, in bytes
template <typename T>
__device__ __forceinline__ void row_load(const T* p, int align, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        if (align >= 16) {
            const uint4 a = mx_ld(reinterpret_cast<const uint4*>(p)), b = mx_ld(reinterpret_cast<const uint4*>(p) + 1);
            v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
            return;
        }
    } else if (align >= 16) {
        const uint4 a = mx_ld(reinterpret_cast<const uint4*>(p));
        const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mx_to_f32(h[e]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = mx_to_f32(mx_ld(p + e));
}

template <typename T>
__device__ __forceinline__ void row_store(T* p, int align, const float (&v)[8]) {
    T h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = mx_from_f32<T>(v[e]);
    if (align >= 16) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(h)[i];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = h[e];
    }
}

// a + b exactly, as the rounded sum and what it lost (Knuth's two-sum)
__device__ __forceinline__ float two_sum(float a, float b, float& lost) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// 1 / sqrt(mean of squares + eps), correctly rounded to fp32 but for about one row in 2^20: what
// 64-bit arithmetic gives, so that a cached code next to a border does not depend on the order of a
// sum.  Sums are kept as two fp32 (the products' and sums' roundings are carried on), about 12
// fp32 operations a value; in fp64, of which this chip does a 64th as many, 8192 tokens' keys would
// take 90 us.  inv_dim: 1 / D as two fp32.  The estimate y of rsqrtf takes one Newton step,
// y - y (a y^2 - 1) / 2, whose residual is computed from the exact square of y.
template <int LANES>
__device__ __forceinline__ float inverse_norm(const float (&v)[8], float2 inv_dim, float eps) {
    float hi = 0.0f, lo = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float p = __fmul_rn(v[e], v[e]);
        float lost;
        hi = two_sum(hi, p, lost);
        lo = __fadd_rn(lo, __fadd_rn(__fmaf_rn(v[e], v[e], -p), lost));
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
        const float h2 = __shfl_xor_sync(0xffffffffu, hi, d), l2 = __shfl_xor_sync(0xffffffffu, lo, d);
        float lost;
        hi = two_sum(hi, h2, lost);
        lo = __fadd_rn(__fadd_rn(lo, l2), lost);
    }
    float lost;
    hi = two_sum(hi, lo, lost);
    lo = lost;
    const float m = __fmul_rn(hi, inv_dim.x);
    const float m_lo = __fmaf_rn(hi, inv_dim.y, __fmaf_rn(lo, inv_dim.x, __fmaf_rn(hi, inv_dim.x, -m)));
    float a = two_sum(m, eps, lost);
    float a_lo = __fadd_rn(lost, m_lo);
    a = two_sum(a, a_lo, lost);
    a_lo = lost;
    const float y = rsqrtf(a), y2 = __fmul_rn(y, y), y2_lo = __fmaf_rn(y, y, -y2);
    const float residual = __fadd_rn(__fmaf_rn(a, y2, -1.0f), __fmaf_rn(a, y2_lo, __fmul_rn(a_lo, y2)));
    return __fmaf_rn(__fmul_rn(-0.5f, y), residual, y);
}

// cosines and sines of a lane's values: pairs (i, i + rot / 2), or (2i, 2i + 1)
struct Turn {
    float c[8], s[8];
    bool turns;
};

// `at`: the lane's first value; row: the position's of a table [.][rot] (rot a multiple of 16)
__device__ __forceinline__ void turn_load(Turn& w, const float* row, int rot, bool halves, int at) {
    w.turns = at < rot;
    const int half = rot / 2;
    if (!w.turns) return;
    if (halves) {
        const bool second = at >= half;
        const int i = second ? at - half : at;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const uint4 c = mx_ld(reinterpret_cast<const uint4*>(row + i + e)), s = mx_ld(reinterpret_cast<const uint4*>(row + half + i + e));
            w.c[e] = __uint_as_float(c.x), w.c[e + 1] = __uint_as_float(c.y), w.c[e + 2] = __uint_as_float(c.z), w.c[e + 3] = __uint_as_float(c.w);
            w.s[e] = __uint_as_float(s.x), w.s[e + 1] = __uint_as_float(s.y), w.s[e + 2] = __uint_as_float(s.z), w.s[e + 3] = __uint_as_float(s.w);
        }
        // the first of a pair takes a c - b s, the second b c + a s
        if (!second)
#pragma unroll
            for (int e = 0; e < 8; ++e) w.s[e] = -w.s[e];
    } else {
        const uint4 c = mx_ld(reinterpret_cast<const uint4*>(row + at / 2)), s = mx_ld(reinterpret_cast<const uint4*>(row + half + at / 2));
        const uint32_t cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w.c[e] = __uint_as_float(cc[e / 2]);
            w.s[e] = e & 1 ? __uint_as_float(ss[e / 2]) : -__uint_as_float(ss[e / 2]);
        }
    }
}

// v = v c + partner s, each product and the sum rounded (so that results do not depend on who
// computes them); `back`: by the opposite angle.  All 32 lanes call it; halves is uniform.
__device__ __forceinline__ void turn(float (&v)[8], const Turn& w, bool halves, int at, int rot, bool back = false) {
    float o[8];
    if (halves) {
        const int lane = threadIdx.x & 31;
        const int from = w.turns ? (at >= rot / 2 ? lane - rot / 16 : lane + rot / 16) : lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, v[e], from);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[e ^ 1];
    }
    if (w.turns)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(__fmul_rn(v[e], w.c[e]), __fmul_rn(o[e], back ? -w.s[e] : w.s[e]));
}

}  // namespace q4q
