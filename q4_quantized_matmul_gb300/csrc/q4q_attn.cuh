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

#include <type_traits>

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

// A lane holds 8 consecutive values of a row as 4 pairs, which the two-lane fp32 instructions take; a row takes LANES
// lanes (8, 16 or 32, D / 8 of them in use), so a warp holds 32 / LANES rows.
struct Row8 {
    uint64_t p[4];
    __device__ __forceinline__ void clear() { p[0] = p[1] = p[2] = p[3] = 0; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(p[i], v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = pack2(v[2 * i], v[2 * i + 1]);
    }
};

// a + b and a - b.  Where a or b is a product the assembler may contract both into one multiply-add (it does, for the two-lane
// forms, whatever their rounding says): only for sums that take no harm from it.
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) { return ffma2(a, pack2(1.0f, 1.0f), b); }
__device__ __forceinline__ uint64_t fsub2(uint64_t a, uint64_t b) { return ffma2(b, pack2(-1.0f, -1.0f), a); }

// what a row's 8 values of a lane are loaded as
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

// 8 values at p; `align`: of every row's start, in bytes
template <typename T>
__device__ __forceinline__ void raw_load(const T* p, int align, Raw8<T>& r) {
    if (align >= 16) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = mx_ld(reinterpret_cast<const uint4*>(p) + i);
    } else {
        uint32_t b[4 * (sizeof(T) / 2)];
#pragma unroll
        for (int i = 0; i < 4 * (int)sizeof(T) / 2; ++i) {
            if constexpr (sizeof(T) == 4) b[i] = mx_ld(reinterpret_cast<const uint32_t*>(p) + i);
            else b[i] = (uint32_t)mx_ld(reinterpret_cast<const uint16_t*>(p) + 2 * i) | (uint32_t)mx_ld(reinterpret_cast<const uint16_t*>(p) + 2 * i + 1) << 16;
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
    }
}
__device__ __forceinline__ void raw_get(const Raw8<float>& r, Row8& v) {
    v.p[0] = (uint64_t)r.w[0].y << 32 | r.w[0].x, v.p[1] = (uint64_t)r.w[0].w << 32 | r.w[0].z;
    v.p[2] = (uint64_t)r.w[1].y << 32 | r.w[1].x, v.p[3] = (uint64_t)r.w[1].w << 32 | r.w[1].z;
}
__device__ __forceinline__ void raw_get(const Raw8<__half>& r, Row8& v) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v.p[i] = pack2(f.x, f.y);
    }
}
__device__ __forceinline__ void raw_get(const Raw8<__nv_bfloat16>& r, Row8& v) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ void row_load(const T* p, int align, float (&v)[8]) {
    Raw8<T> r;
    raw_load(p, align, r);
    Row8 x;
    raw_get(r, x);
    x.get(v);
}

template <typename T>
__device__ __forceinline__ void row_store(T* p, int align, const Row8& x) {
    float v[8];
    x.get(v);
    if (align >= 16) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same_v<T, __half>) {
                    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = mx_from_f32<T>(v[e]);
    }
}

// a + b exactly, as the rounded sum and what it lost (Knuth's two-sum)
__device__ __forceinline__ float two_sum(float a, float b, float& lost) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// 1 / sqrt(mean of squares + eps) of 4 rows, of which a lane holds 8 values each, correctly rounded to fp32 but for
// about one row in 2^20: what 64-bit arithmetic gives, so that a cached code next to a border does not depend on the
// order of a sum.  Sums are kept as two fp32 (what the squares' and sums' roundings lose is carried on); fp64, of which
// this chip does a 64th as many, would take 90 us for 8192 tokens' keys.  The lanes of a row halve the rows among them
// in the first two steps of the sum, so that each ends with one row's, takes its root and hands it round.  inv_dim:
// 1 / D as two fp32.  The estimate y of rsqrtf takes one Newton step, y - y (a y^2 - 1) / 2, whose residual
// is computed from the exact product a y, which is in range wherever a is (y^2 as two fp32 is not: of means past 2^112 its lower part was
// subnormal, and up to 2% of rows one rounding off).  EXACT: squares of 16-bit values are exact in fp32.  (A square contracted into its
// sum changes that sum by at most its own rounding, which the two-sum then carries on.)
template <int LANES, bool EXACT>
__device__ __forceinline__ void inverse_norm4(const Row8 (&v)[4], float2 inv_dim, float eps, float (&r)[4]) {
    const int lane = threadIdx.x & 31;
    float hi[4], lo[4], lost;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint64_t h = 0, l = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t p = fmul2(v[n].p[i], v[n].p[i]);
            if constexpr (!EXACT) l = fadd2(l, ffma2(v[n].p[i], v[n].p[i], fmul2(p, pack2(-1.0f, -1.0f))));
            if (i == 0) {
                h = p;
            } else {
                const uint64_t s = fadd2(h, p), bb = fsub2(s, h);
                l = fadd2(l, fadd2(fsub2(h, fsub2(s, bb)), fsub2(p, bb)));
                h = s;
            }
        }
        float h0, h1, l0, l1;
        unpack2(h, h0, h1);
        unpack2(l, l0, l1);
        hi[n] = two_sum(h0, h1, lost);
        lo[n] = __fadd_rn(__fadd_rn(l0, l1), lost);
    }
    int d = LANES / 2;
    bool upper = lane & d;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float h2 = __shfl_xor_sync(0xffffffffu, upper ? hi[n] : hi[n + 2], d), l2 = __shfl_xor_sync(0xffffffffu, upper ? lo[n] : lo[n + 2], d);
        hi[n] = two_sum(upper ? hi[n + 2] : hi[n], h2, lost);
        lo[n] = __fadd_rn(__fadd_rn(upper ? lo[n + 2] : lo[n], l2), lost);
    }
    d /= 2;
    upper = lane & d;
    float h = upper ? hi[1] : hi[0], l = upper ? lo[1] : lo[0];
    {
        const float h2 = __shfl_xor_sync(0xffffffffu, upper ? hi[0] : hi[1], d), l2 = __shfl_xor_sync(0xffffffffu, upper ? lo[0] : lo[1], d);
        h = two_sum(h, h2, lost);
        l = __fadd_rn(__fadd_rn(l, l2), lost);
    }
#pragma unroll
    for (d /= 2; d > 0; d /= 2) {
        const float h2 = __shfl_xor_sync(0xffffffffu, h, d), l2 = __shfl_xor_sync(0xffffffffu, l, d);
        h = two_sum(h, h2, lost);
        l = __fadd_rn(__fadd_rn(l, l2), lost);
    }
    h = two_sum(h, l, lost);
    l = lost;
    const float m = __fmul_rn(h, inv_dim.x);
    const float m_lo = __fmaf_rn(h, inv_dim.y, __fmaf_rn(l, inv_dim.x, __fmaf_rn(h, inv_dim.x, -m)));
    float a = two_sum(m, eps, lost);
    float a_lo = __fadd_rn(lost, m_lo);
    a = two_sum(a, a_lo, lost);
    a_lo = lost;
    const float y = rsqrtf(a), ay = __fmul_rn(a, y), ay_lo = __fmaf_rn(a, y, -ay);
    const float residual = __fadd_rn(__fmaf_rn(ay, y, -1.0f), __fmaf_rn(ay_lo, y, __fmul_rn(__fmul_rn(a_lo, y), y)));
    const float mine = __fmaf_rn(__fmul_rn(-0.5f, y), residual, y);
#pragma unroll
    for (int n = 0; n < 4; ++n) r[n] = __shfl_sync(0xffffffffu, mine, (lane & ~(LANES - 1)) | (n & 2 ? LANES / 2 : 0) | (n & 1 ? LANES / 4 : 0));
}

// Cosines and sines of a lane's values: pairs (i, i + rot / 2), or (2i, 2i + 1).  Of a pair (a, b) the first becomes
// a c - b s, the second b c + a s: s has its sign here.
struct Turn {
    Row8 c, s;
    int from;           // the lane that holds the partners (pairs of halves)
    bool turns;
};

__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) { return (uint64_t)y << 32 | x; }

// What does not depend on the position; `at`: the lane's first value, rot a multiple of 16.
__device__ __forceinline__ void turn_init(Turn& w, int rot, bool halves, int at) {
    const int lane = threadIdx.x & 31;
    w.turns = at < rot;
    w.from = halves && w.turns ? (at >= rot / 2 ? lane - rot / 16 : lane + rot / 16) : lane;
    w.c.clear();
    w.s.clear();
}

// row: the position's of a table [.][rot]; back: the opposite angle
__device__ __forceinline__ void turn_load(Turn& w, const float* row, int rot, bool halves, int at, bool back) {
    if (!w.turns) return;
    const int half = rot / 2;
    if (halves) {
        const bool second = at >= half;
        const uint4* c = reinterpret_cast<const uint4*>(row + (second ? at - half : at));
        const uint4 c0 = mx_ld(c), c1 = mx_ld(c + 1), s0 = mx_ld(c + half / 4), s1 = mx_ld(c + half / 4 + 1);
        const uint32_t flip = second != back ? 0u : 0x80000000u;
        w.c.p[0] = pair_of(c0.x, c0.y), w.c.p[1] = pair_of(c0.z, c0.w), w.c.p[2] = pair_of(c1.x, c1.y), w.c.p[3] = pair_of(c1.z, c1.w);
        w.s.p[0] = pair_of(s0.x ^ flip, s0.y ^ flip), w.s.p[1] = pair_of(s0.z ^ flip, s0.w ^ flip);
        w.s.p[2] = pair_of(s1.x ^ flip, s1.y ^ flip), w.s.p[3] = pair_of(s1.z ^ flip, s1.w ^ flip);
    } else {
        const uint4 c = mx_ld(reinterpret_cast<const uint4*>(row + at / 2)), s = mx_ld(reinterpret_cast<const uint4*>(row + half + at / 2));
        const uint32_t first = back ? 0u : 0x80000000u, second = back ? 0x80000000u : 0u;
        w.c.p[0] = pair_of(c.x, c.x), w.c.p[1] = pair_of(c.y, c.y), w.c.p[2] = pair_of(c.z, c.z), w.c.p[3] = pair_of(c.w, c.w);
        w.s.p[0] = pair_of(s.x ^ first, s.x ^ second), w.s.p[1] = pair_of(s.y ^ first, s.y ^ second);
        w.s.p[2] = pair_of(s.z ^ first, s.z ^ second), w.s.p[3] = pair_of(s.w ^ first, s.w ^ second);
    }
}

// v = v c + partner s, each product and the sum rounded (so that results do not depend on who computes them).  All 32
// lanes call it; halves is uniform.
__device__ __forceinline__ void turn(Row8& v, const Turn& w, bool halves) {
    Row8 o;
    if (halves) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o.p[i] = pair_of(__shfl_sync(0xffffffffu, (uint32_t)v.p[i], w.from), __shfl_sync(0xffffffffu, (uint32_t)(v.p[i] >> 32), w.from));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = pair_of((uint32_t)(v.p[i] >> 32), (uint32_t)v.p[i]);
    }
    if (w.turns)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x0, x1, y0, y1;
            unpack2(fmul2(v.p[i], w.c.p[i]), x0, x1);
            unpack2(fmul2(o.p[i], w.s.p[i]), y0, y1);
            v.p[i] = pack2(__fadd_rn(x0, y0), __fadd_rn(x1, y1));
        }
}

}  // namespace q4q
