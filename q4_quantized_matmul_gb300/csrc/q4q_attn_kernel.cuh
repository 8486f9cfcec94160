// q4q_attn_kernel.cuh -- attention over the paged 4-bit cache on warp-level MMAs: few rows of queries
// a key-value head, and every case that needs fp32 through and through.  q4q_attn_d*.cu instantiate it.
//
// Of query row i and key-value head h, over the keys j that the row sees:
//   s_j = scale <q_i, K_j>,  o_i = sum_j exp(s_j) V_j / sum_j exp(s_j)
// in one pass over the cache with the running maximum m and sum l of the softmax (base 2: the scale
// takes log2 e along).  With K = (code - 8) d by blocks of 32 dims, V likewise:
//   s_j = sum_b dk_jb (sum_{c in b} q_c (code_jc - 8)),  o = sum_j (p_j dv_jb) (code_jc - 8)
// so codes are exact integers in m16n8k16 MMAs with fp32 sums; the keys' scales multiply the sums of
// a block, the values' scales the weights p, and neither is ever rounded.  The codes are the operand of
// 16 rows (16 keys, then 16 dims), the queries the one of 8 columns:
//   S^T [16 keys, 8] = K [16 keys, 32 of a block] q^T,   O^T [16 dims, 8] += V^T [16 dims, 16 keys] P^T
// A lane's sums of S are keys g, g + 8 and columns 2t, 2t + 1; scaled and packed to fp16, an 8 x 8 transposition
// (movmatrix) makes them the operand of the second product.
//  - SPLIT: columns 0-3 hold the high, 4-7 the low fp16 half of 4 queries, and of their weights, so that both
//    count with 22 bits; else 8 queries, exact as fp16 of a power of two times their row, weights rounded
//    to fp16 (2^-12, less than a bf16 result's rounding by 2^3).
//  - CENTRED: key codes become code - 8 in fp16 (9 operations for 8 codes).  Else they are taken as they are, a
//    nibble as a fp16 subnormal, code 2^-24, or 16 times that where it lies in a byte's upper half, whose q was
//    divided by 16, and -8 sum q is what the sum starts from (5 operations for 8).  The tensor cores align a
//    subnormal by its nominal exponent, which costs about 7 bits: scores are good to 1e-5.
//    Value codes are always centred: an offset left in sums over many keys would be far larger than they.
//  - Weights are p = exp2(s - r).  r is a row's: it makes the largest product p dv so far 2^7 to 2^15, which is what goes into
//    the second MMA.  A block of 32 dims whose products are below 2^2 there has a unit of its own, a power of two u that p dv u is taken
//    with, so that a product counts to 2^-27 of the largest of its row and block, whatever values other blocks or rows have, or keys without
//    weight.  (One exponent for a warp, of the largest scale of any key, left scales 2^10 below that 2.4e-3 from 64 bits.)
//    Every step a lane compares its largest score and scale with 2^15, and a vote over the warp finds where one is past it; only then
//    r and u move and sums are rescaled: by the largest score where the step's scales are near each other, else by the products
//    themselves.  r is a score less a whole number: that key's weight is a power of two, its product exact.  (64 bf16 tokens over 8192
//    keys at most: 96 us with the one exponent, 98 so; 101 with the products looked at each time, 109 with units read in every step.)
//
// Work.  All steps (two chunks of 16 tokens of a head, 2304 bytes each at D = 128) of all pieces -- a sequence, head and
// tile of rows -- in a row are cut into equal shares, one a CTA, two CTAs an SM, so a ragged batch or one long
// sequence both fill the GPU.  A producer warp's 32 lanes each find and copy one chunk in 32 (a bulk copy into a
// ring of steps), the consumer warps take the steps in turn.  At the end of a piece its consumers' sums are joined in
// shared memory; what a CTA leaves of a piece to others goes to the workspace as sums with r and l, and
// a second kernel joins the parts in order.
//
// Measured in a graph (heads 32/8 of 128): one fp32 token over 1023 keys 14.0 us (launches, shares, a piece's end and the
// join); over 131072 keys, fp16, 47 us (151 MB, 3.2 TB/s); 64 bf16 tokens over 8192 keys at most 98 us (337 MB, 3.4 TB/s).
// Some 300 instructions a chunk of 16 keys and warp, issued in 55% of the cycles, the ALU pipe busy in half of them, HBM at half its rate:
// no unit is full, four warps a scheduler leave the rest to latency.  (32 to 72 bytes of spills in one group's forms at D = 128, 450 to 650 in two
// groups' at D = 256.)
#pragma once

#include <algorithm>
#include <type_traits>

#include "q4q_attn.cuh"
#include "q4q_attn_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_attn_status = 0;

constexpr int STEP = 2 * KV_GROUP;        // tokens that a warp takes at a time: two chunks

constexpr float NONE = -1e30f;           // the reference of a row that has seen no key: exp2(-inf - NONE) is 0

// What a type of queries is computed as.
enum Kind { KIND_F32, KIND_F16, KIND_BF16 };

template <int B_, int KIND, int NG_>
struct Cfg {
    static constexpr int B = B_;                       // blocks of 32 dims
    static constexpr int NG = NG_;                     // groups of 8 columns
    static constexpr bool SPLIT = KIND != KIND_BF16;
    static constexpr bool CENTRED = KIND == KIND_F32;
    using T = std::conditional_t<KIND == KIND_F32, float, std::conditional_t<KIND == KIND_F16, __half, __nv_bfloat16>>;
    static constexpr int ROWS = (SPLIT ? 4 : 8) * NG;  // of a tile
    static constexpr int DIM = 32 * B;
    static constexpr int CHUNK = kv_chunk_bytes(DIM);
    // Two CTAs of 8 warps an SM where 128 registers are nearly enough (8 B for the sums of a group of columns, 4 B for its
    // queries; B = 4 spills up to 72 bytes), so that one's end of a piece hides behind the other's chunks.
    static constexpr int CTAS = B <= 4 && NG == 1 ? 2 : 1;
    static constexpr int CONSUMERS = 7;
    static constexpr int THREADS = (CONSUMERS + 1) * 32;
    // Slots of a step each.  A slot is always the same warp's: one that took another's could run a round ahead of it and
    // mistake the phase before for its own.
    static constexpr int PER_WARP = B > 4 && NG == 2 ? 1 : 2;
    static constexpr int SLOTS = PER_WARP * CONSUMERS;
    static constexpr int OUT_STRIDE = DIM + 4;         // of a row of a warp's sums: conflict-free
    static constexpr int BARS = 0;                     // full, then empty
    static constexpr int META = BARS + 2 * SLOTS * 8;  // [SLOTS][2]: 1 for a chunk that is not there
    static constexpr int MISC = META + SLOTS * 8;      // scan and broadcast words
    static constexpr int STOP = MISC + 248;            // the abort flag
    static constexpr int STATS = MISC + 256;           // [CONSUMERS][ROWS] reference and sum
    static constexpr int UNITS = STATS + CONSUMERS * ROWS * 8;   // [CONSUMERS][2][NG][B][4 t] two fp32, of columns 2t, 2t + 1: units, what sums are multiplied by
    static constexpr int RING = (UNITS + CONSUMERS * NG * B * 64 + 127) / 128 * 128;
    static constexpr int OUT = RING + SLOTS * 2 * CHUNK;
    static constexpr int BYTES = OUT + CONSUMERS * ROWS * OUT_STRIDE * 4;
    static_assert(SLOTS <= 16, "a lane of the producer for each half of a slot");
    static_assert(MISC % 8 == 0 && CHUNK % 16 == 0 && OUT % 16 == 0, "alignment of copies and vectors");
    static_assert(BYTES * CTAS <= (227 - CTAS) * 1024, "shared memory of an SM");
};

// What a worker left in the workspace: a part of a segment (sequence, head, tile), its steps from .. to - 1
// of `of`.
struct Part {
    int seq, head, tile;
    int from, to, of;
};

// The workspace: parts [2 * workers], then of each ROWS x D sums and their references and sums.
struct Plan {
    Part* parts;
    float* rows;
    int workers;
    int least;            // steps a worker should have at least
    int whole;            // 1: a piece is never cut
};

// A sequence's rows and keys.
struct Seq {
    int q0, n, len;       // first row, rows, cached tokens
    int tiles;            // of TILE_ROWS rows (tokens x shared heads)
    int cost;             // steps that a tile is counted as
};

template <int TILE_ROWS>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int s, bool whole) {
    Seq r;
    if (a.first) {
        const int64_t f0 = mx_ld(a.first + s), f1 = mx_ld(a.first + s + 1);
        r.q0 = (int)min(max(f0, (int64_t)0), a.n_q);
        r.n = (int)(min(max(f1, (int64_t)r.q0), a.n_q) - r.q0);
    } else {
        r.q0 = s;
        r.n = s < a.n_q ? 1 : 0;
    }
    const int64_t most = a.max_pages << a.page_log;
    const int l = mx_ld(a.kv_len + s);
    if ((l < 0 || l > most) && threadIdx.x % 32 == 0) record_error(&g_attn_status, Q4Q_ERR_ARG);
    r.len = (int)min(max((int64_t)l, (int64_t)0), most);
    r.tiles = (int)(((int64_t)r.n * a.shared + TILE_ROWS - 1) / TILE_ROWS);
    int64_t keys = r.len;
    if (a.window > 0) keys = min(keys, a.window + TILE_ROWS + STEP);  // a tile's rows are at most as many tokens
    r.cost = whole ? 1 : max(1, (int)((keys + STEP - 1) / STEP));
    return r;
}

__device__ __forceinline__ int64_t units_of(const AttnArgs& a, const Seq& s) { return (int64_t)s.tiles * a.kv_heads * s.cost; }

// row / shared
__device__ __forceinline__ int divided(int row, const AttnArgs& a) { return a.shared == 1 ? row : (int)(__umulhi((uint32_t)row, a.shared_m) >> a.shared_s); }

// The keys that row `row` (token * shared + head) of a sequence sees: [lo, hi).
__device__ __forceinline__ void keys_of(const AttnArgs& a, const Seq& s, int row, int& lo, int& hi) {
    const int64_t last = a.causal ? (int64_t)s.len - s.n + divided(row, a) : (int64_t)s.len - 1;
    hi = (int)max(last + 1, (int64_t)0);
    lo = a.window > 0 ? (int)max(last + 1 - a.window, (int64_t)0) : 0;
    if (lo > hi) lo = hi;
}

// A walk over a worker's units [at, end): pieces, one after another.
struct Walk {
    int64_t at, end, base;     // base: the first unit of sequence s
    int s;
    Seq seq;
    int head, tile, from, to;  // the piece
    int g0, g1;                // its steps: g0 .. g1 - 1 of the sequence
    bool valid;
};

template <int TILE_ROWS>
__device__ __forceinline__ void next_piece(const AttnArgs& a, Walk& w, bool whole) {
    w.valid = false;
    while (w.at < w.end) {
        const int64_t units = units_of(a, w.seq);
        if (w.at - w.base >= units) {
            w.base += units;
            ++w.s;
            w.seq = seq_of<TILE_ROWS>(a, w.s, whole);
            continue;
        }
        const uint32_t cost = (uint32_t)w.seq.cost;
        const int64_t rel = w.at - w.base;
        const int64_t segment = rel / cost;
        w.from = (int)(rel - segment * cost);
        w.to = (int)min((int64_t)cost, w.from + (w.end - w.at));
        w.head = (int)(segment / w.seq.tiles);
        w.tile = (int)(segment - (int64_t)w.head * w.seq.tiles);
        w.at += w.to - w.from;
        // the tile's steps, and this piece's of them
        int lo, hi, unused;
        keys_of(a, w.seq, w.tile * TILE_ROWS, lo, unused);
        keys_of(a, w.seq, min(w.tile * TILE_ROWS + TILE_ROWS, w.seq.n * a.shared) - 1, unused, hi);
        const int c0 = lo / STEP, c1 = (hi + STEP - 1) / STEP;
        w.g0 = whole ? c0 : min(c0 + w.from, c1);
        w.g1 = whole ? c1 : min(c0 + w.to, c1);
        w.valid = true;
        return;
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                        float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// an 8 x 8 matrix of 16-bit values turned over, two values a lane
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// what the fp16 pair h leaves of x and y, as fp16
__device__ __forceinline__ uint32_t rest2(float x, float y, uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return half2_bits(x - f.x, y - f.y);
}

template <int WORDS>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&v)[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]) : "r"(addr + i * 4));
    } else if constexpr (WORDS % 2 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i]), "=r"(v[i + 1]) : "r"(addr + i * 4));
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[i]) : "r"(addr + i * 4));
    }
}

// B fp16 scales of a token, two a word
template <int B>
__device__ __forceinline__ void lds_scales(uint32_t addr, uint32_t (&v)[(B + 1) / 2]) {
    if constexpr (B % 2 == 0) {
        lds<B / 2>(addr, v);
    } else {
        uint16_t h[B];
#pragma unroll
        for (int i = 0; i < B; ++i) asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h[i]) : "r"(addr + i * 2));
#pragma unroll
        for (int i = 0; i < (B + 1) / 2; ++i) v[i] = h[2 * i] | (2 * i + 1 < B ? (uint32_t)h[2 * i + 1] << 16 : 0u);
    }
}

template <int W>
__device__ __forceinline__ float scale_at(const uint32_t (&w)[W], int i) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[i >> 1]);
    return i & 1 ? __high2float(h) : __low2float(h);
}

// 2^e as fp32, -126 <= e <= 127
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// of a normal number above 0
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// Products with a row's reference and a block's unit are at most UNIT_MOST; where they move they make the largest at least
// 2^UNIT_BITS.  Weights are at most 2^WEIGHT_BITS (of rows whose values are all 0, or next to it).
constexpr int UNIT_BITS = 7, WEIGHT_BITS = 90;
constexpr float UNIT_MOST = 32768.0f, UNIT_LEAST = 4.0f;
__device__ __forceinline__ void pair_load(uint32_t addr, float& x, float& y) {
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x), "=f"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ float word_load(uint32_t addr) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void word_store(uint32_t addr, float x) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory"); }

// the larger of the magnitudes of two fp16 pairs (a NaN gives way)
__device__ __forceinline__ uint32_t largest2(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)), __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// whether the phase is complete, without the wait that try_wait may take
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

template <typename T>
__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, float4 v) {
    T* p = static_cast<T*>(a.dst) + at;
    if constexpr (sizeof(T) == 4) {
        if (a.align >= 16) *reinterpret_cast<float4*>(p) = v;
        else p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    } else {
        const T h0 = mx_from_f32<T>(v.x), h1 = mx_from_f32<T>(v.y), h2 = mx_from_f32<T>(v.z), h3 = mx_from_f32<T>(v.w);
        if (a.align >= 16) {
            auto bits = [](T lo, T hi) { return (uint32_t)reinterpret_cast<const uint16_t&>(lo) | (uint32_t)reinterpret_cast<const uint16_t&>(hi) << 16; };
            *reinterpret_cast<uint2*>(p) = make_uint2(bits(h0, h1), bits(h2, h3));
        } else {
            p[0] = h0, p[1] = h1, p[2] = h2, p[3] = h3;
        }
    }
}

// The share of a part with reference r in sums whose reference is R (none where r is -inf; a NaN stays)
__device__ __forceinline__ float share_of(float r, float R) { return r == -INFINITY ? 0.0f : exp2f(r - R); }
__device__ __forceinline__ float larger(float x, float y) { return x != x || y != y ? NAN : fmaxf(x, y); }

// One worker's units and what it is to write down of them.
struct Share {
    int64_t u0, u1, base;
    int s;
};

// All units, this worker's share of them, and the sequence that it starts in: every thread takes a
// run of sequences, the block adds them up.  `words`: WARPS + 2 words of shared memory.
template <int THREADS, int TILE_ROWS>
__device__ __forceinline__ Share share_of_worker(const AttnArgs& a, const Plan& plan, int64_t* words) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.n_seqs + THREADS - 1) / THREADS, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
    int64_t sum = 0;
    for (int s = s0; s < s1; ++s) sum += units_of(a, seq_of<TILE_ROWS>(a, s, plan.whole));
    int64_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) words[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += words[w];
        total += words[w];
    }
    const int64_t workers = min((int64_t)plan.workers, max((int64_t)1, total / plan.least));
    Share r;
    r.u0 = min(total, (total * blockIdx.x + workers - 1) / workers);
    r.u1 = blockIdx.x >= workers ? r.u0 : min(total, (total * (blockIdx.x + 1) + workers - 1) / workers);
    if (blockIdx.x >= workers) r.u0 = r.u1 = total;
    // the thread whose run holds the first unit walks to its sequence
    if (r.u0 < r.u1 && before <= r.u0 && r.u0 < before + sum) {
        int s = s0;
        while (true) {
            const int64_t n = units_of(a, seq_of<TILE_ROWS>(a, s, plan.whole));
            if (r.u0 < before + n) break;
            before += n;
            ++s;
        }
        words[WARPS] = before;
        words[WARPS + 1] = s;
    }
    __syncthreads();
    r.base = words[WARPS];
    r.s = (int)words[WARPS + 1];
    return r;
}

// The producer warp: its lanes find the chunks of the next SLOTS steps, one each (lane 2 i + h: half h of step i), and
// copy each when its slot is free.
constexpr int AHEAD = 7;

template <typename C>
__device__ __forceinline__ void produce(const AttnArgs& a, const Plan& plan, Walk w, uint32_t base, uint8_t* smem) {
    const int lane = threadIdx.x & 31, in_page = a.page_log - 4, step = lane >> 1;
    volatile int* stop = reinterpret_cast<volatile int*>(smem + C::STOP);
    const uint32_t full = base + C::BARS + step * 8, empty = full + C::SLOTS * 8;
    bool skip_copy = a.fault && blockIdx.x == 0 && lane == 0;
    int used = 0;                                    // steps of the piece that are handled
    uint32_t phase = 0;                              // copies made into this lane's half slot
    bool ok = true;
    next_piece<C::ROWS>(a, w, plan.whole);
    while (w.valid) {
        bool mine = false;
        int s = 0, head = 0, group = 0, filled = 0, groups = 0;
        while (w.valid && filled < C::SLOTS) {
            const int n = min(w.g1 - w.g0 - used, C::SLOTS - filled);
            if (step >= filled && step < filled + n) {
                mine = true;
                s = w.s;
                head = w.head;
                group = 2 * (w.g0 + used + step - filled) + (lane & 1);
                groups = (w.seq.len + KV_GROUP - 1) / KV_GROUP;
            }
            filled += n;
            used += n;
            if (used == w.g1 - w.g0) {
                next_piece<C::ROWS>(a, w, plan.whole);
                used = 0;
            }
        }
        // the second half of a sequence's last step may lie behind its last token
        int page = -1;
        if (mine && group < groups) page = mx_ld(a.pages + s * a.max_pages + (group >> in_page));
        const bool there = page >= 0 && page < a.n_pages;
        if (mine && group < groups && !there) record_error(&g_attn_status, Q4Q_ERR_ARG);
        const uint8_t* from = a.cache + kv_chunk_offset(there ? page : 0, head, group & ((1 << in_page) - 1), a.kv_heads, a.page_log, C::DIM);
        uint32_t open = __ballot_sync(0xffffffffu, mine);
        while (open) {
            // Wait for one of the next slots that are still to be filled, not for each of them: they are freed in about this
            // order.  (One that is filled already would be waited for in vain, where its step is of a piece behind this one's.)
            const int next = 31 - __clz(open & (0xffffffffu >> (31 - min(__ffs(open) - 1 + AHEAD, 31))));
            const uint32_t its = __shfl_sync(0xffffffffu, phase, next), bar = __shfl_sync(0xffffffffu, empty, next);
            if (its > 0) {
                const bool free = mbar_try_wait(bar, (its - 1) & 1) || mbar_wait_until(bar, (its - 1) & 1, stop, a.limit_ns);
                if (!__all_sync(0xffffffffu, free)) {
                    ok = false;
                    break;
                }
            }
            if (mine && (phase == 0 || mbar_test(empty, (phase - 1) & 1))) {
                reinterpret_cast<volatile int*>(smem + C::META)[lane] = !there;
                if (there) {
                    mbar_arrive_expect_tx(full, C::CHUNK);
                    if (!skip_copy) bulk_g2s(base + C::RING + lane * C::CHUNK, from, C::CHUNK, full);
                } else {
                    mbar_arrive(full);
                }
                skip_copy = false;
                ++phase;
                mine = false;
            }
            open = __ballot_sync(0xffffffffu, mine);
        }
        if (!ok) break;
    }
    if (!ok) *stop = 1;
    // copies in flight must land before this CTA's shared memory is another's: consumers that gave up leave some
    if (phase > 0) mbar_wait_bounded(full, (phase - 1) & 1, a.limit_ns);
    __syncwarp();
}

template <typename C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS) attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    constexpr int B = C::B, NG = C::NG, CONSUMERS = C::CONSUMERS, W = (B + 1) / 2;
    using T = typename C::T;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    volatile int* stop = reinterpret_cast<volatile int*>(smem + C::STOP);
    if (tid < 2 * C::SLOTS) mbar_init(base + C::BARS + tid * 8, tid < C::SLOTS ? 2 : 1);
    if (tid == 0) *stop = 0;
    fence_mbar_init();
    pdl_trigger();
    pdl_wait();
    // what is copied below may have been written by ordinary stores of the work before
    asm volatile("fence.proxy.async;" ::: "memory");
    const Share share = share_of_worker<C::THREADS, C::ROWS>(a, plan, reinterpret_cast<int64_t*>(smem + C::MISC));
    if (tid < 2 && !plan.whole) plan.parts[2 * blockIdx.x + tid].of = -1;
    if (share.u0 >= share.u1) return;
    Walk work;
    work.at = share.u0;
    work.end = share.u1;
    work.base = share.base;
    work.s = share.s;
    work.seq = seq_of<C::ROWS>(a, work.s, plan.whole);
    if (warp == CONSUMERS) {
        produce<C>(a, plan, work, base, smem);
        return;
    }

    const uint32_t units = base + C::UNITS + warp * NG * B * 64 + t * 8, downs = units + NG * B * 32;     // + (q * B + b) * 32
    float2* stats = reinterpret_cast<float2*>(smem + C::STATS);
    float* out = reinterpret_cast<float*>(smem + C::OUT);
    int numbered = 0;                                // steps of this CTA before the piece's
    int taken = 0;                                   // steps of this warp: the CTA's every CONSUMERS-th
    bool dead = false;                               // a wait ran out: the rest is passed over
    while (true) {
        next_piece<C::ROWS>(a, work, plan.whole);
        if (!work.valid) break;
        const Seq& seq = work.seq;
        const int rows = seq.n * a.shared, tile0 = work.tile * C::ROWS, steps = work.g1 - work.g0;

        // The queries' operand.  Lane (g, t) holds column g's dims 32 b + 8 t .. + 7, scaled by a power of two so that the
        // row's largest is in [2^14, 2^15), in the order of the codes' nibbles: (0, 4), (1, 5), (2, 6), (3, 7).
        uint32_t qf[NG][B][4];
        uint32_t off[NG][2];                         // -8 sum q of each block, in two fp16: blocks 2t, 2t + 1 of column g
        float row_scale[NG][2];
        int lo[NG][2], hi[NG][2];                    // keys that this lane's columns 2t, 2t + 1 see
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const int row = min(tile0 + (C::SPLIT ? q * 4 + (g & 3) : q * 8 + g), rows - 1);
            const T* from = static_cast<const T*>(a.q) + (int64_t)(seq.q0 + row / a.shared) * a.q_stride +
                            (int64_t)(work.head * a.shared + row % a.shared) * C::DIM + 8 * t;
            float v[B][8];
            float top = 0.0f, off_low = 0.0f;
            off[q][0] = off[q][1] = 0u;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                row_load(from + 32 * b, a.align, v[b]);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[b][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 100);
            const float up = two_to(14 - e);
            // back from 2^(14 - e), and with codes taken as subnormals from their 2^-24
            const float mine = a.scale_log2 * two_to(C::CENTRED ? e - 14 : e + 10);
            row_scale[q][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
            row_scale[q][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
#pragma unroll
            for (int b = 0; b < B; ++b) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[b][k] *= up;
                if constexpr (!C::CENTRED) {
                    float sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum += v[b][k];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    sum *= C::SPLIT && g >= 4 ? 0.0f : -8.0f * 5.9604644775390625e-8f;   // 2^-24
                    if (b % 2 == 0) off_low = sum;
                    if ((b % 2 == 1 || b == B - 1) && t == b / 2) {
                        off[q][0] = half2_bits(off_low, b % 2 ? sum : 0.0f);
                        off[q][1] = rest2(off_low, b % 2 ? sum : 0.0f, off[q][0]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float less = !C::CENTRED && k % 2 ? 0.0625f : 1.0f;
                    const float x = v[b][k] * less, y = v[b][k + 4] * less;
                    const uint32_t h = half2_bits(x, y);
                    qf[q][b][k] = C::SPLIT && g >= 4 ? rest2(x, y, h) : h;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                keys_of(a, seq, min(tile0 + (C::SPLIT ? q * 4 + ((2 * t + i) & 3) : q * 8 + 2 * t + i), rows - 1), lo[q][i], hi[q][i]);
        }
        int lo_all = lo[0][0], hi_all = hi[0][0];    // seen by every row of the tile
#pragma unroll
        for (int q = 0; q < NG; ++q) lo_all = max(lo_all, max(lo[q][0], lo[q][1])), hi_all = min(hi_all, min(hi[q][0], hi[q][1]));
        lo_all = __reduce_max_sync(0xffffffffu, lo_all);
        hi_all = __reduce_min_sync(0xffffffffu, hi_all);

        float o[NG][B][2][4];
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[q][b][i / 4][i % 4] = 0.0f;
        float ref[NG][2], l[NG][2];                  // of columns 2t, 2t + 1; l: this lane's sum
#pragma unroll
        for (int q = 0; q < NG; ++q) ref[q][0] = ref[q][1] = NONE, l[q][0] = l[q][1] = 0.0f;
        bool mixed = false;                          // some block of some row has a unit of its own

        const int start = warp + CONSUMERS * taken - numbered;
        for (int i = start; i < steps && !dead; i += CONSUMERS, ++taken) {
            const uint32_t slot = warp + CONSUMERS * (taken % C::PER_WARP), parity = (taken / C::PER_WARP) & 1;
            const uint32_t full = base + C::BARS + slot * 8, chunk = base + C::RING + slot * 2 * C::CHUNK;
            const bool ok = mbar_try_wait(full, parity) || mbar_wait_until(full, parity, stop, a.limit_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                dead = true;
                if (lane == 0) {
                    if (!*stop) record_error(&g_attn_status, DEV_TIMEOUT);
                    *stop = 1;
                }
                break;
            }
            uint32_t gone[2];                        // chunks that are not there
            lds<2>(base + C::META + slot * 8, gone);
            const int key0 = (work.g0 + i) * STEP;
            const bool edge = key0 < lo_all || key0 + STEP > hi_all || (gone[0] | gone[1]);

            // scores of keys g + 8 j and columns 2t, 2t + 1
            float y[NG][8];
            uint32_t dv[4][W];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = chunk + h * C::CHUNK;
                uint32_t w[2][B], dk[2][W];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lds<B>(at + (j * 32 + lane) * 4 * B, w[j]);
                    lds_scales<B>(at + 16 * C::DIM + (j * 8 + g) * 2 * B, dk[j]);
                    lds_scales<B>(at + 17 * C::DIM + (j * 8 + g) * 2 * B, dv[2 * h + j]);
                }
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    float first[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if constexpr (!C::CENTRED) {
                        // sum_b d_b (-8 sum q): 8 blocks deep, the high and the low halves of the sums
                        uint32_t d[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            d[j] = t & 1 ? dk[j][1 % W] : dk[j][0];
                            if constexpr (W > 2) d[j] = t & 2 ? (t & 1 ? dk[j][3 % W] : dk[j][2 % W]) : d[j];
                        }
                        mma_f16(first, d[0], d[1], d[0], d[1], off[q][0], off[q][1], 0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[q][4 * h + k] = first[k];
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    uint32_t c[2][4];                // codes of key g, g + 8: nibbles (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (C::CENTRED) {
                            const uint4 x = nibbles_to_f16x8(w[j][b]);
                            c[j][0] = x.x, c[j][1] = x.y, c[j][2] = x.z, c[j][3] = x.w;
                        } else {
                            const uint32_t w8 = w[j][b] >> 8;
                            c[j][0] = w[j][b] & 0x000F000Fu, c[j][1] = w[j][b] & 0x00F000F0u, c[j][2] = w8 & 0x000F000Fu, c[j][3] = w8 & 0x00F000F0u;
                        }
                    }
                    const float d0 = scale_at(dk[0], b), d1 = scale_at(dk[1], b);
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        float acc[4];
                        mma_f16(acc, c[0][0], c[1][0], c[0][1], c[1][1], qf[q][b][0], qf[q][b][1], 0.0f, 0.0f, 0.0f, 0.0f);
                        mma_f16(acc, c[0][2], c[1][2], c[0][3], c[1][3], qf[q][b][2], qf[q][b][3]);
                        float* z = y[q] + 4 * h;
                        z[0] = fmaf(acc[0], d0, z[0]), z[1] = fmaf(acc[1], d0, z[1]);
                        z[2] = fmaf(acc[2], d1, z[2]), z[3] = fmaf(acc[3], d1, z[3]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (C::SPLIT) y[q][k] += __shfl_xor_sync(0xffffffffu, y[q][k], 2);
                    y[q][k] *= row_scale[q][k & 1];
                }
            bool careful = false;
            if (edge) {
                // keys that a row does not see, and the scales of slots that no row does
                uint32_t odd = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + 8 * j + g;
                    const bool lost = gone[j / 2];
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        if (key < lo[q][0] || key >= hi[q][0] || lost) y[q][2 * j] = -INFINITY;
                        if (key < lo[q][1] || key >= hi[q][1] || lost) y[q][2 * j + 1] = -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        if (key >= seq.len || lost) dv[j][k] = 0u;
                        odd |= __vcmpgtu2(dv[j][k] & 0x7FFF7FFFu, 0x7BFF7BFFu);
                    }
                }
                // a scale that is no number, in a step that not every row sees: weights of 0 have to stay 0
                careful = __any_sync(0xffffffffu, odd != 0);
            }
            float x[NG][8], top[NG][2];
#pragma unroll
            for (int q = 0; q < NG; ++q) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[q][k] = y[q][k] - ref[q][k & 1];
#pragma unroll
                for (int c = 0; c < 2; ++c) top[q][c] = fmaxf(fmaxf(x[q][c], x[q][2 + c]), fmaxf(x[q][4 + c], x[q][6 + c]));
            }
            float most = top[0][0];
#pragma unroll
            for (int q = 0; q < NG; ++q) most = fmaxf(most, fmaxf(top[q][0], top[q][1]));
            uint32_t dm[W];                                                        // each block's largest scale of this lane's keys
#pragma unroll
            for (int k = 0; k < W; ++k) dm[k] = largest2(largest2(dv[0][k], dv[1][k]), largest2(dv[2][k], dv[3][k]));
            uint32_t bits = dm[0];
#pragma unroll
            for (int k = 1; k < W; ++k) bits = __vmaxu2(bits, dm[k]);
            bits = max(bits >> 16, bits & 0xFFFFu);
            bool past = most > (float)min(29 - (int)(bits >> 10), WEIGHT_BITS);    // a scale is below 2^(exponent field - 14)
            if (mixed) {
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        float u[2];
                        pair_load(units + (q * B + b) * 32, u[0], u[1]);
#pragma unroll
                        for (int c = 0; c < 2; ++c) past |= ex2(top[q][c]) * scale_at(dm, b) * u[c] > UNIT_MOST;
                    }
            }
            if (__any_sync(0xffffffffu, past)) {
                // Where no scale of the step's keys is further than 2^5 below the largest, the key of a row's largest score has products of 2^2
                // to 2^8 in every block once r is that score less 8 and more the largest scale's exponent.
                uint32_t low = 0x7BFF7BFFu, high = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool there = key0 + 8 * j + g < seq.len && !gone[j / 2];
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        const uint32_t d = dv[j][k] & 0x7FFF7FFFu;
                        high = __vmaxu2(high, d);
                        if (there) low = __vminu2(low, B % 2 && k == W - 1 ? d | 0x7BFF0000u : d);
                    }
                }
                low = __reduce_min_sync(0xffffffffu, min(low >> 16, low & 0xFFFFu)) >> 10;
                high = __reduce_max_sync(0xffffffffu, max(high >> 16, high & 0xFFFFu)) >> 10;
                if (!mixed && high < 31 && low > 0 && low + 5 >= high) {
                    const int e = (int)high - 14;                                  // scales are below 2^e
#pragma unroll
                    for (int q = 0; q < NG; ++q)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float n = fmaxf(fmaxf(y[q][c], y[q][2 + c]), fmaxf(y[q][4 + c], y[q][6 + c]));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
                            const float old = ref[q][c], now = n - old > (float)(UNIT_BITS + 8 - e) ? n - (float)(UNIT_BITS + 1 - e) : old;
                            const float down = ex2(old - now);
                            l[q][c] *= down;
                            ref[q][c] = now;
#pragma unroll
                            for (int b = 0; b < B; ++b) o[q][b][0][c] *= down, o[q][b][0][2 + c] *= down, o[q][b][1][c] *= down, o[q][b][1][2 + c] *= down;
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[q][2 * j + c] = y[q][2 * j + c] - now;
                        }
                } else {
                    // The products themselves, of column c and block b the largest of the warp's keys: lanes g = 2 (b % 4) + c share them out.
                    // An infinite or NaN scale makes its own dims so, and says nothing about the others'.
                    bool own = false;
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        constexpr int SETS = (B + 3) / 4;                              // of 4 blocks
                        float n[2], w[8], v[SETS][8];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            n[c] = fmaxf(fmaxf(y[q][c], y[q][2 + c]), fmaxf(y[q][4 + c], y[q][6 + c]));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) n[c] = fmaxf(n[c], __shfl_xor_sync(0xffffffffu, n[c], d));
#pragma unroll
                            for (int j = 0; j < 4; ++j) w[2 * j + c] = ex2(y[q][2 * j + c] - (n[c] == -INFINITY ? 0.0f : n[c]));
                        }
                        float all = 0.0f;                                              // the row's largest product, over 2^n
#pragma unroll
                        for (int k = 0; k < SETS; ++k) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                v[k][i] = 0.0f;
                                if (4 * k + i / 2 < B)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        const float d = fabsf(scale_at(dv[j], 4 * k + i / 2));
                                        if (d <= 65504.0f) v[k][i] = fmaxf(v[k][i], w[2 * j + i % 2] * d);
                                    }
                            }
#pragma unroll
                            for (int d = 4; d > 0; d >>= 1)
#pragma unroll
                                for (int i = 0; i < d; ++i) {
                                    const float other = __shfl_xor_sync(0xffffffffu, g & d ? v[k][i] : v[k][i + d], 4 * d);
                                    v[k][i] = fmaxf(g & d ? v[k][i + d] : v[k][i], other);
                                }
                            all = fmaxf(all, v[k][0]);
                        }
                        all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, 8));
                        all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, 16));
                        // of this lane's column
                        const float most_y = g & 1 ? n[1] : n[0], old = g & 1 ? ref[q][1] : ref[q][0];
                        const bool none = old == NONE;                                 // no sums yet
                        float now = old;
                        if (most_y > -INFINITY && (none || most_y - old > (float)WEIGHT_BITS || all * ex2(most_y - old) > UNIT_MOST))
                            now = most_y - (float)min(UNIT_BITS - exponent_of(all), WEIGHT_BITS);
                        const float by = none ? 0.0f : now - old, whole = floorf(by), scale = ex2(most_y - now);
#pragma unroll
                        for (int k = 0; k < SETS; ++k) {
                            const int b = 4 * k + (g >> 1);
                            if (b < B) {
                                const uint32_t at = (q * B + b) * 32 + (g & 1) * 4;
                                // As it was, if it can: the block's sums keep their bits.  At most WEIGHT_BITS more than the row's.
                                const int was = none || !mixed ? 0 : exponent_of(word_load(units + at)), kept = none ? WEIGHT_BITS : min(was + (int)fminf(whole, 1000.0f), WEIGHT_BITS);
                                const float product = v[k][0] * scale;
                                const int unit = now == NONE || product >= UNIT_LEAST ? 0 : product * two_to(kept) > UNIT_MOST ? UNIT_BITS - exponent_of(product) : kept;
                                word_store(units + at, two_to(unit));
                                word_store(downs + at, none ? 1.0f : ex2(whole - by) * two_to(max(unit - was - (int)fminf(whole, 1000.0f), -126)));
                                own |= unit != 0;
                            }
                        }
                        const float now2[2] = {__shfl_sync(0xffffffffu, now, t), __shfl_sync(0xffffffffu, now, 4 + t)};
                        __syncwarp();
#pragma unroll
                        for (int b = 0; b < B; ++b) {
                            float down[2];
                            pair_load(downs + (q * B + b) * 32, down[0], down[1]);
#pragma unroll
                            for (int c = 0; c < 2; ++c) o[q][b][0][c] *= down[c], o[q][b][0][2 + c] *= down[c], o[q][b][1][c] *= down[c], o[q][b][1][2 + c] *= down[c];
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            l[q][c] *= ex2(ref[q][c] - now2[c]);
                            ref[q][c] = now2[c];
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[q][2 * j + c] = y[q][2 * j + c] - now2[c];
                        }
                    }
                    mixed = __any_sync(0xffffffffu, own);
                }
            }
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[q][k] = ex2(x[q][k]);                                        // from here the weight
                    l[q][k & 1] += x[q][k];
                }
            const auto values = [&](auto of_care) {                               // of_care: units, and scales that are no numbers
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[2][B];
#pragma unroll
                    for (int j = 0; j < 2; ++j) lds<B>(chunk + h * C::CHUNK + 8 * C::DIM + (j * 32 + lane) * 4 * B, w[j]);
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const float d0 = scale_at(dv[2 * h], b), d1 = scale_at(dv[2 * h + 1], b);
                        const uint4 c0 = nibbles_to_f16x8(w[0][b]), c1 = nibbles_to_f16x8(w[1][b]);
#pragma unroll
                        for (int q = 0; q < NG; ++q) {
                            const float* z = x[q] + 4 * h;
                            float p[4] = {z[0] * d0, z[1] * d0, z[2] * d1, z[3] * d1};
                            if constexpr (decltype(of_care)::value) {
                                float u[2];
                                if (mixed) pair_load(units + (q * B + b) * 32, u[0], u[1]);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if (mixed) p[k] *= u[k & 1];
                                    if (y[q][4 * h + k] == -INFINITY) p[k] = 0.0f;
                                }
                            }
                            uint32_t p0 = half2_bits(p[0], p[1]), p1 = half2_bits(p[2], p[3]);
                            if constexpr (C::SPLIT) {
                                const uint32_t r0 = rest2(p[0], p[1], p0), r1 = rest2(p[2], p[3], p1);
                                p0 = t < 2 ? p0 : r0;
                                p1 = t < 2 ? p1 : r1;
                            }
                            p0 = transposed(p0);
                            p1 = transposed(p1);
                            mma_f16(o[q][b][0], c0.x, c0.y, c1.x, c1.y, p0, p1);
                            mma_f16(o[q][b][1], c0.z, c0.w, c1.z, c1.w, p0, p1);
                        }
                    }
                }
            };
            if (careful || mixed) values(std::true_type{});
            else values(std::false_type{});
            __syncwarp();                            // the step is read by all lanes before it is written again
            if (lane == 0) mbar_arrive(full + C::SLOTS * 8);
        }
        numbered += steps;

        // Join the warps: of column 2t + c this lane's dims 32 b + 4 g .. + 3, its reference and sum.
        const bool any = start < steps;
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float sum = l[q][c];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = C::SPLIT ? q * 4 + 2 * (t & 1) + c : q * 8 + 2 * t + c;
                // scores that are all NaN leave no maximum, but a NaN in the sum
                if (g == 0 && (!C::SPLIT || t < 2))
                    stats[warp * C::ROWS + row] = make_float2(any && (ref[q][c] != NONE || sum != 0.0f) ? ref[q][c] : -INFINITY, sum);
                if (any)
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const float u = mixed ? two_to(-exponent_of(word_load(units + (q * B + b) * 32 + c * 4))) : 1.0f;
                        float4 v = make_float4(o[q][b][0][c] * u, o[q][b][0][2 + c] * u, o[q][b][1][c] * u, o[q][b][1][2 + c] * u);
                        if constexpr (C::SPLIT) {
                            v.x += __shfl_xor_sync(0xffffffffu, v.x, 2), v.y += __shfl_xor_sync(0xffffffffu, v.y, 2);
                            v.z += __shfl_xor_sync(0xffffffffu, v.z, 2), v.w += __shfl_xor_sync(0xffffffffu, v.w, 2);
                        }
                        if (!C::SPLIT || t < 2) *reinterpret_cast<float4*>(out + (warp * C::ROWS + row) * C::OUT_STRIDE + 32 * b + 4 * g) = v;
                    }
            }
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
        const bool complete = work.from == 0 && work.to == seq.cost;
        const int part = 2 * blockIdx.x + (work.from == 0 ? 1 : 0);
        float* part_rows = plan.rows + (int64_t)part * (C::ROWS * (C::DIM + 2));
        if (!complete && tid == 0) plan.parts[part] = {work.s, work.head, work.tile, work.from, work.to, seq.cost};
        for (int i = tid; i < C::ROWS * (C::DIM / 4); i += CONSUMERS * 32) {
            const int r = i / (C::DIM / 4), c = i % (C::DIM / 4) * 4;
            if (tile0 + r >= rows) break;                                          // r grows with i
            float2 st[CONSUMERS];
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < CONSUMERS; ++w) {
                st[w] = stats[w * C::ROWS + r];
                top = larger(top, st[w].x);
            }
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < CONSUMERS; ++w) {
                if (st[w].x == -INFINITY) continue;                                // nothing was written there
                const float k = exp2f(st[w].x - top);
                const float4 x = *reinterpret_cast<const float4*>(out + (w * C::ROWS + r) * C::OUT_STRIDE + c);
                sum = fmaf(k, st[w].y, sum);
                v.x = fmaf(k, x.x, v.x), v.y = fmaf(k, x.y, v.y), v.z = fmaf(k, x.z, v.z), v.w = fmaf(k, x.w, v.w);
            }
            if (complete) {
                const float inv = top == -INFINITY ? 0.0f : 1.0f / sum;
                const int64_t at = (int64_t)(seq.q0 + (tile0 + r) / a.shared) * a.heads + work.head * a.shared + (tile0 + r) % a.shared;
                store4<T>(a, at * C::DIM + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (c == 0 && a.lse) a.lse[at] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
            } else {
                *reinterpret_cast<float4*>(part_rows + r * C::DIM + c) = v;
                if (c == 0) *reinterpret_cast<float2*>(part_rows + C::ROWS * C::DIM + 2 * r) = make_float2(top, sum);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
    }
}

// Joins the parts of the segments that were cut.  A segment's parts are a worker's last one (its
// start) and the first ones of the workers behind it; block (w, r) joins row r of the one that starts
// in worker w.
constexpr int JOIN_WARPS = 8, JOIN_AT_ONCE = 4;   // a warp takes every 8th part, 4 of them in flight

template <typename C>
__global__ void __launch_bounds__(JOIN_WARPS * 32) join_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    constexpr int VEC = C::DIM / 32;
    __shared__ float sums[JOIN_WARPS][C::DIM];
    __shared__ float shares[JOIN_WARPS];
    pdl_wait();
    const int w = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Part* parts = plan.parts;
    const int of = mx_ld(&parts[2 * w + 1].of), to0 = mx_ld(&parts[2 * w + 1].to);
    if (of < 0 || to0 >= of) return;                       // no segment starts here, or none that goes on
    const int s = mx_ld(&parts[2 * w + 1].seq), head = mx_ld(&parts[2 * w + 1].head), tile = mx_ld(&parts[2 * w + 1].tile);
    // the workers behind: whose first part ends the segment
    int n = 1;
    for (bool more = true; more; n += 32) {
        const int v = w + n + lane;
        const bool goes_on = v < plan.workers && mx_ld(&parts[2 * v].of) >= 0 && mx_ld(&parts[2 * v].to) < of;
        const uint32_t ends = __ballot_sync(0xffffffffu, !goes_on);
        more = !ends;
        if (ends) n += __ffs(ends) - 32;
    }
    n = min(n, plan.workers - w);
    const Seq seq = seq_of<C::ROWS>(a, s, plan.whole);
    const int row = tile * C::ROWS + r;
    if (row >= seq.n * a.shared) return;
    const auto rows_of = [&](int p) { return plan.rows + (p == 0 ? 2 * w + 1 : 2 * (w + p)) * (int64_t)(C::ROWS * (C::DIM + 2)); };
    // the largest reference first: all of them in flight together
    float ref = -INFINITY;
    for (int p = lane; p < n; p += 32) ref = larger(ref, mx_ld(rows_of(p) + C::ROWS * C::DIM + 2 * r));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ref = larger(ref, __shfl_xor_sync(0xffffffffu, ref, d));
    float sum = 0.0f, v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
    for (int p0 = warp; p0 < n; p0 += JOIN_WARPS * JOIN_AT_ONCE) {
        float k[JOIN_AT_ONCE], l[JOIN_AT_ONCE], x[JOIN_AT_ONCE][VEC];
#pragma unroll
        for (int q = 0; q < JOIN_AT_ONCE; ++q) {
            const float* rows = rows_of(min(p0 + q * JOIN_WARPS, n - 1));
            k[q] = mx_ld(rows + C::ROWS * C::DIM + 2 * r);
            l[q] = mx_ld(rows + C::ROWS * C::DIM + 2 * r + 1);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] = mx_ld(rows + r * C::DIM + i * 32 + lane);
        }
#pragma unroll
        for (int q = 0; q < JOIN_AT_ONCE; ++q) {
            if (p0 + q * JOIN_WARPS >= n) break;
            const float share = share_of(k[q], ref);
            sum = fmaf(share, l[q], sum);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = fmaf(share, x[q][i], v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) sums[warp][i * 32 + lane] = v[i];
    if (lane == 0) shares[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < JOIN_WARPS; ++x) sum += shares[x];
    const float inv = ref == -INFINITY ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t)(seq.q0 + row / a.shared) * a.heads + head * a.shared + row % a.shared;
    for (int c = threadIdx.x * 4; c < C::DIM; c += JOIN_WARPS * 128) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < JOIN_WARPS; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(&sums[i][c]);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        store4<typename C::T>(a, at * C::DIM + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    }
    if (threadIdx.x == 0 && a.lse) a.lse[at] = ref == -INFINITY ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <typename K, typename... Args>
q4q_status launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? launch_status() : (cudaGetLastError(), Q4Q_ERR_CUDA);
}

template <typename C>
q4q_status run(const AttnArgs& a, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    const cudaError_t e = cudaFuncSetAttribute(attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return cudaGetLastError(), Q4Q_ERR_CUDA;
    Plan plan;
    plan.workers = info.sm_count * C::CTAS;
    plan.whole = (a.max_pages << a.page_log) <= STEP * C::CONSUMERS;
    plan.least = plan.whole ? 1 : C::CONSUMERS;
    plan.parts = static_cast<Part*>(workspace);
    plan.rows = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + mx_up((int64_t)sizeof(Part) * 2 * plan.workers, 256));
    const q4q_status st = launch(attn_kernel<C>, dim3((unsigned)plan.workers), C::THREADS, C::BYTES, stream, a, plan);
    if (st != Q4Q_OK || plan.whole) return st;
    return launch(join_kernel<C>, dim3((unsigned)plan.workers, C::ROWS), JOIN_WARPS * 32, 0, stream, a, plan);
}

template <typename C>
size_t workspace_of(const DeviceInfo& info) {
    const int64_t workers = (int64_t)info.sm_count * C::CTAS;
    return (size_t)(mx_up((int64_t)sizeof(Part) * 2 * workers, 256) + (int64_t)sizeof(float) * C::ROWS * (C::DIM + 2) * 2 * workers);
}

// that of the forms with the most rows
template <int B>
size_t attn_workspace(const DeviceInfo& info) {
    return std::max(workspace_of<Cfg<B, KIND_BF16, 1>>(info), workspace_of<Cfg<B, KIND_BF16, 2>>(info));
}

// `wide`: two groups of columns
template <int B>
q4q_status attn_run(const AttnArgs& a, bool wide, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    switch (a.type) {
        case Q4Q_TYPE_F32: return wide ? run<Cfg<B, KIND_F32, 2>>(a, workspace, stream, info) : run<Cfg<B, KIND_F32, 1>>(a, workspace, stream, info);
        case Q4Q_TYPE_F16: return wide ? run<Cfg<B, KIND_F16, 2>>(a, workspace, stream, info) : run<Cfg<B, KIND_F16, 1>>(a, workspace, stream, info);
        default: return wide ? run<Cfg<B, KIND_BF16, 2>>(a, workspace, stream, info) : run<Cfg<B, KIND_BF16, 1>>(a, workspace, stream, info);
    }
}

unsigned int attn_take_status_word() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_attn_status, &z, sizeof(z));
    return v;
}

}  // namespace
}  // namespace q4q
