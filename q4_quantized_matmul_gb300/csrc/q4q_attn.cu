// q4q_attn.cu -- attention over the paged 4-bit cache: few rows of queries a key-value head, and
// every case that needs fp32 through and through.
//
// Of query row i and key-value head h, over the keys j that the row sees:
//   s_j = scale <q_i, K_j>,  o_i = sum_j exp(s_j) V_j / sum_j exp(s_j)
// in one pass over the cache with the running maximum m and sum l of the softmax (base 2: the scale
// takes log2 e along).  With K = (code - 8) d by blocks of 32 dims, V likewise:
//   s_j = sum_b dk_jb (sum_{c in b} q_c code_jc - 8 sum_{c in b} q_c)
//   o   = sum_j (p_j dv_jb) (code_jc - 8)
// so codes are the exact integer operands of m16n8k16 MMAs with fp32 sums, the keys' scales multiply
// the sums of a block, the values' scales the weights p, and neither is ever rounded.  The other operand
// has 8 rows (queries of the head's group, and of several tokens): rows 0-7 of the MMA hold its high,
// rows 8-15 its low fp16 half, so queries and weights count with 22 bits at no further MMA.
//  - Key codes go to the tensor cores as they are: a nibble is a fp16 subnormal, code 2^-24, or 16
//    times that where it lies in a byte's upper half, whose q was divided by 16.  5 operations for 8.
//  - Value codes become code - 8 as fp16 (9 operations for 8): with the codes' offset of 8 left in the
//    sums, those would be far larger than their difference where many keys weigh alike.
//  - Weights are exp2(s - m - E + 8) with E the largest exponent of the values' scales so far: p dv is
//    at most 2^8, and m and E move only when something passes them by 2^6, which a vote over
//    the warp finds; sums are rescaled only then.
//
// Work.  A warp takes 16 tokens at a time: one bulk copy of a chunk (2304 bytes at D = 128) into
// its own ring of shared memory, waited for on its own barrier, no hand-off between warps.  A CTA's
// warps take every WARPS-th chunk of a piece: a sequence, head and tile of 8 rows, or a part of its
// chunks.  All pieces' chunks in a row are cut into equal shares, one for each CTA (one an SM), so a
// ragged batch or one long sequence both fill the GPU; what a CTA leaves of a piece to others goes
// to the workspace as sums with m and l, and a second kernel joins the parts in order.
#include <algorithm>

#include "q4q_attn.cuh"
#include "q4q_attn_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_attn_status = 0;

constexpr int ROWS = 8;                  // rows of a tile

template <int B>
struct Shape {
    static constexpr int DIM = 32 * B;
    static constexpr int CHUNK = kv_chunk_bytes(DIM);
    static constexpr int WARPS = B <= 4 ? 12 : 8;
    static constexpr int STAGES = B <= 4 ? 4 : 3;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int OUT_STRIDE = DIM + 4;                                    // of a row of a warp's sums: conflict-free
    static constexpr bool Q_SHARED = B > 4;                                       // the queries' operand registers in shared memory
    static constexpr int BARS = 0;
    static constexpr int MISC = BARS + WARPS * STAGES * 8;                        // scan and broadcast words
    static constexpr int STATS = MISC + 512;                                      // [WARPS][ROWS] reference and sum
    static constexpr int RING = (STATS + WARPS * ROWS * 8 + 127) / 128 * 128;
    static constexpr int OUT = RING + WARPS * STAGES * CHUNK;
    static constexpr int QF = OUT + WARPS * ROWS * OUT_STRIDE * 4;
    static constexpr int BYTES = QF + (Q_SHARED ? B * 2 * 32 * 16 : 0);
    static_assert(RING % 128 == 0 && CHUNK % 16 == 0 && OUT % 16 == 0 && QF % 16 == 0, "alignment of copies and vectors");
    static_assert(BYTES <= 227 * 1024, "shared memory of an SM");
};

// What a worker left in the workspace: a part of segment `segment` (sequence, head, tile), chunks
// [from, to) of `of`.
struct Part {
    int seq, head, tile;
    int from, to, of;
};

// rows of a part: sums [8][D], then reference and sum of each row
template <int B>
__host__ __device__ constexpr int64_t part_floats() { return ROWS * Shape<B>::DIM + 2 * ROWS; }

// The workspace: parts [2 * workers], then their rows.
struct Plan {
    Part* parts;
    float* rows;
    int workers;
    int least;            // chunks a worker should have at least
    int whole;            // 1: a piece is never cut
};

// A sequence's rows and keys.
struct Seq {
    int q0, n, len;       // first row, rows, cached tokens
    int tiles;            // of ROWS rows (tokens x shared heads)
    int cost;             // chunks that a tile is counted as
};

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
    r.tiles = (int)(((int64_t)r.n * a.shared + ROWS - 1) / ROWS);
    int64_t keys = r.len;
    if (a.window > 0) keys = min(keys, a.window + ROWS + KV_GROUP);       // a tile's rows are at most ROWS tokens
    r.cost = whole ? 1 : max(1, (int)((keys + KV_GROUP - 1) / KV_GROUP));
    return r;
}

__device__ __forceinline__ int64_t units_of(const AttnArgs& a, const Seq& s) { return (int64_t)s.tiles * a.kv_heads * s.cost; }

// The keys that row `row` (token * shared + head) of a sequence sees: [lo, hi).
__device__ __forceinline__ void keys_of(const AttnArgs& a, const Seq& s, int row, int& lo, int& hi) {
    const int64_t last = a.causal ? (int64_t)s.len - s.n + row / a.shared : (int64_t)s.len - 1;
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
    int g0, g1;                // its chunks: g0 .. g1 - 1 of the sequence
    bool valid;
};

__device__ __forceinline__ void next_piece(const AttnArgs& a, Walk& w, bool whole) {
    w.valid = false;
    while (w.at < w.end) {
        const int64_t units = units_of(a, w.seq);
        if (w.at - w.base >= units) {
            w.base += units;
            ++w.s;
            w.seq = seq_of(a, w.s, whole);
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
        // the tile's chunks, and this piece's of them
        int lo, hi, unused;
        keys_of(a, w.seq, w.tile * ROWS, lo, unused);
        keys_of(a, w.seq, min(w.tile * ROWS + ROWS, w.seq.n * a.shared) - 1, unused, hi);
        const int c0 = lo / KV_GROUP, c1 = (hi + KV_GROUP - 1) / KV_GROUP;
        w.g0 = whole ? c0 : min(c0 + w.from, c1);
        w.g1 = whole ? c1 : min(c0 + w.to, c1);
        w.valid = true;
        return;
    }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x and y as fp16 pairs: the nearest, and what they leave
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
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

// 2^e as fp32, -126 <= e <= 127
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// half i of the scales of two tokens [2][B], as they lie
template <int B>
__device__ __forceinline__ float scale_at(const uint32_t (&w)[B], int i) {
    return fp16_to_f32(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
}

// 8 values of a row of q, any type
__device__ __forceinline__ void load_q(const AttnArgs& a, int64_t at, float (&v)[8]) {
    switch (a.type) {
        case Q4Q_TYPE_F32: row_load(static_cast<const float*>(a.q) + at, a.align, v); break;
        case Q4Q_TYPE_F16: row_load(static_cast<const __half*>(a.q) + at, a.align, v); break;
        default: row_load(static_cast<const __nv_bfloat16*>(a.q) + at, a.align, v); break;
    }
}

__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, float4 v) {
    if (a.type == Q4Q_TYPE_F32) {
        float* p = static_cast<float*>(a.dst) + at;
        if (a.align >= 16) *reinterpret_cast<float4*>(p) = v;
        else p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
        return;
    }
    uint2 u;
    if (a.type == Q4Q_TYPE_F16) {
        const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
        u = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        u = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    uint16_t* p = static_cast<uint16_t*>(a.dst) + at;
    if (a.align >= 16) *reinterpret_cast<uint2*>(p) = u;
    else p[0] = (uint16_t)u.x, p[1] = (uint16_t)(u.x >> 16), p[2] = (uint16_t)u.y, p[3] = (uint16_t)(u.y >> 16);
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
// run of sequences, the block adds them up.  `words`: 64 bytes x 8 of shared memory.
template <int THREADS>
__device__ __forceinline__ Share share_of_worker(const AttnArgs& a, const Plan& plan, int64_t* words) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.n_seqs + THREADS - 1) / THREADS, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
    int64_t sum = 0;
    for (int s = s0; s < s1; ++s) sum += units_of(a, seq_of(a, s, plan.whole));
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
            const int64_t n = units_of(a, seq_of(a, s, plan.whole));
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

template <int B>
__global__ void __launch_bounds__(Shape<B>::THREADS, 1) attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    using S = Shape<B>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t bars = base + S::BARS + warp * S::STAGES * 8;
    const uint32_t ring = base + S::RING + warp * S::STAGES * S::CHUNK;
    float2* stats = reinterpret_cast<float2*>(smem + S::STATS);
    if (lane == 0)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(bars + i * 8, 1);
    fence_mbar_init();
    pdl_trigger();
    pdl_wait();
    // what is copied below may have been written by ordinary stores of the work before
    asm volatile("fence.proxy.async;" ::: "memory");
    const Share share = share_of_worker<S::THREADS>(a, plan, reinterpret_cast<int64_t*>(smem + S::MISC));
    if (tid < 2 && !plan.whole) plan.parts[2 * blockIdx.x + tid].of = -1;
    if (share.u0 >= share.u1) return;

    // The warp's chunks in order: `load` walks ahead of `work` by up to STAGES of them.
    Walk work;
    work.at = share.u0;
    work.end = share.u1;
    work.base = share.base;
    work.s = share.s;
    work.seq = seq_of(a, work.s, plan.whole);
    Walk load = work;
    next_piece(a, load, plan.whole);
    int next = load.g0 + warp;                       // the chunk to copy next
    int page = -1;                                   // its page, looked up a step before its copy
    bool dead = false;                               // a wait ran out
    uint32_t issued = 0, taken = 0;                  // copies
    uint32_t looked = 0, passed = 0, absent = 0;     // chunks; bit i of absent: chunk i (mod 32) has no page
    bool skip_copy = a.fault && blockIdx.x == 0 && warp == 0;
    const int in_page = a.page_log - 4;
    auto look_up = [&]() {
        while (load.valid && next >= load.g1) {
            next_piece(a, load, plan.whole);
            next = load.g0 + warp;
        }
        if (load.valid) page = mx_ld(a.pages + load.s * a.max_pages + (next >> in_page));
    };
    look_up();
    // one copy; a page that is not there gives none, and is passed over below in the same way
    auto copy = [&]() {
        if (!load.valid) return;
        if (page >= 0 && page < a.n_pages) {
            if (lane == 0) {
                const uint32_t bar = bars + (issued % S::STAGES) * 8;
                mbar_arrive_expect_tx(bar, S::CHUNK);
                if (!skip_copy)
                    bulk_g2s(ring + (issued % S::STAGES) * S::CHUNK,
                             a.cache + kv_chunk_offset(page, load.head, next & ((1 << in_page) - 1), a.kv_heads, a.page_log, S::DIM), S::CHUNK, bar);
            }
            skip_copy = false;
            ++issued;
            absent &= ~(1u << (looked & 31));
        } else {
            absent |= 1u << (looked & 31);
        }
        ++looked;
        next += S::WARPS;
        look_up();
    };
    for (int i = 0; i < S::STAGES; ++i) copy();

    while (true) {
        next_piece(a, work, plan.whole);
        if (!work.valid) break;
        const Seq& seq = work.seq;
        const int rows = seq.n * a.shared, tile0 = work.tile * ROWS;

        // The queries: lane (g, t) holds row g's dims 32 b + 8 t .. + 7, scaled so that the row's largest is
        // in [2^14, 2^15), in the order of the MMA's operand: (0, 4), (1, 5) / 16 and (2, 6), (3, 7) / 16.
        const int row = min(tile0 + g, rows - 1);
        const int token = row / a.shared, head = work.head * a.shared + row % a.shared;
        const int64_t q_at = (int64_t)(seq.q0 + token) * a.q_stride + (int64_t)head * S::DIM + 8 * t;
        int lo, hi;
        keys_of(a, seq, row, lo, hi);
        const int lo_all = __reduce_max_sync(0xffffffffu, lo), hi_all = __reduce_min_sync(0xffffffffu, hi);   // seen by every row
        uint32_t qf[S::Q_SHARED ? 1 : B][2][4];
        float off[B];
        float row_scale;
        {
            float v[B][8];
            float top = 0.0f;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                load_q(a, q_at + 32 * b, v[b]);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[b][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 100);
            const float up = two_to(14 - e);
            row_scale = a.scale_log2 * two_to(e + 10);                            // 2^(e - 14) and the codes' 2^24
            if constexpr (S::Q_SHARED) __syncthreads();                           // the operand of the piece before is done with
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[b][k] *= up;
                    sum += v[b][k];
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                off[b] = -8.0f * 5.9604644775390625e-8f * sum;                    // 2^-24
                uint32_t f[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    split2(v[b][2 * k], v[b][2 * k + 4], f[k][0], f[k][1]);
                    split2(v[b][2 * k + 1] * 0.0625f, v[b][2 * k + 5] * 0.0625f, f[k][2], f[k][3]);
                }
                if constexpr (S::Q_SHARED) {
                    if (b % S::WARPS == warp)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4*>(smem + S::QF + ((b * 2 + k) * 32 + lane) * 16) = make_uint4(f[k][0], f[k][1], f[k][2], f[k][3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r) qf[b][k][r] = f[k][r];
                }
            }
            if constexpr (S::Q_SHARED) __syncthreads();
        }

        float o[B][4][4];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[b][n][r] = 0.0f;
        float m = -INFINITY, l = 0.0f;       // of row g: the maximum that weights refer to; this lane's share of the sum
        int top_e = -32;                     // E: exponents of the values' scales are below it

        for (int c = work.g0 + warp; c < work.g1; c += S::WARPS) {
            if (dead) continue;
            if ((absent >> (passed++ & 31)) & 1) {
                if (lane == 0) record_error(&g_attn_status, Q4Q_ERR_ARG);
                copy();
                continue;
            }
            const uint32_t slot = taken % S::STAGES, bar = bars + slot * 8, chunk = ring + slot * S::CHUNK;
            const bool ok = mbar_try_wait(bar, (taken / S::STAGES) & 1) || mbar_wait_bounded(bar, (taken / S::STAGES) & 1, a.limit_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                dead = true;                 // the rest of this warp's chunks is passed over
                if (lane == 0) record_error(&g_attn_status, DEV_TIMEOUT);
                continue;
            }
            const int key0 = c * KV_GROUP;
            const bool edge = key0 < lo_all || key0 + KV_GROUP > hi_all;

            float s[2][2];
            uint32_t dv[2][B];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[B], dk[B];
                lds<B>(chunk + (j * 32 + lane) * 4 * B, w);
                lds<B>(chunk + 16 * S::DIM + (j * 4 + t) * 4 * B, dk);
                lds<B>(chunk + 17 * S::DIM + (j * 4 + t) * 4 * B, dv[j]);
                s[j][0] = s[j][1] = 0.0f;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    float acc[4] = {off[b], off[b], 0.0f, 0.0f};
                    const uint32_t w8 = w[b] >> 8;
                    uint32_t f[2][4];
                    if constexpr (S::Q_SHARED) {
                        lds<4>(base + S::QF + ((b * 2) * 32 + lane) * 16, f[0]);
                        lds<4>(base + S::QF + ((b * 2 + 1) * 32 + lane) * 16, f[1]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int r = 0; r < 4; ++r) f[k][r] = qf[b][k][r];
                    }
                    mma_f16(acc, f[0][0], f[0][1], f[0][2], f[0][3], w[b] & 0x000F000Fu, w[b] & 0x00F000F0u);
                    mma_f16(acc, f[1][0], f[1][1], f[1][2], f[1][3], w8 & 0x000F000Fu, w8 & 0x00F000F0u);
                    s[j][0] = fmaf(acc[0] + acc[2], scale_at<B>(dk, b), s[j][0]);
                    s[j][1] = fmaf(acc[1] + acc[3], scale_at<B>(dk, B + b), s[j][1]);
                }
                s[j][0] *= row_scale;
                s[j][1] *= row_scale;
            }
            if (edge) {
                // keys that row g does not see, and the scales of slots that no row does
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int key = key0 + 8 * j + 2 * t;
                    if (key < lo || key >= hi) s[j][0] = -INFINITY;
                    if (key + 1 < lo || key + 1 >= hi) s[j][1] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        if (key >= seq.len) dv[j][i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
                        if (key + 1 >= seq.len) dv[j][(B + i) / 2] &= (B + i) % 2 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
                }
            }
            // the values' scales: their largest exponent
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < B; ++i) bits = __vmaxu2(bits, __vmaxu2(dv[0][i] & 0x7FFF7FFFu, dv[1][i] & 0x7FFF7FFFu));
            bits = max(bits >> 16, bits & 0xFFFFu);
            const int above = (int)(bits >> 10) - 14;                              // d < 2^above
            const float top = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            if (__any_sync(0xffffffffu, top > m + 6.0f || above > top_e)) {
                // an infinite or NaN scale makes its own dims so, and says nothing about the others'
                uint32_t finite = 0;
#pragma unroll
                for (int i = 0; i < 2 * B; ++i) {
                    const uint32_t x = dv[i / B][i % B] & 0x7FFF7FFFu;
                    finite = max(finite, max(x >> 16 < 0x7C00u ? x >> 16 : 0u, (x & 0xFFFFu) < 0x7C00u ? x & 0xFFFFu : 0u));
                }
                const int e = max(top_e, (int)(__reduce_max_sync(0xffffffffu, finite) >> 10) - 14);
                float n = fmaxf(m, top);
                n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 1));
                n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2));
                const float down = m == -INFINITY ? 0.0f : exp2f((m - n) + (float)(top_e - e));
                m = n;
                top_e = e;
                l *= down;
#pragma unroll
                for (int b = 0; b < B; ++b)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[b][k][r] *= down;
            }
            const float ref = m + (float)(top_e - 8);
            float p[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    p[j][i] = s[j][i] == -INFINITY ? 0.0f : exp2f(s[j][i] - ref);
                    l += p[j][i];
                }
            uint32_t w[2][B];
#pragma unroll
            for (int j = 0; j < 2; ++j) lds<B>(chunk + 8 * S::DIM + (j * 32 + lane) * 4 * B, w[j]);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                uint32_t pf[4];
                float x[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        x[j][i] = p[j][i] * scale_at<B>(dv[j], i * B + b);
                        if (edge && s[j][i] == -INFINITY) x[j][i] = 0.0f;          // its scale may be anything
                    }
                split2(x[0][0], x[0][1], pf[0], pf[1]);
                split2(x[1][0], x[1][1], pf[2], pf[3]);
                const uint4 c0 = nibbles_to_f16x8(w[0][b]), c1 = nibbles_to_f16x8(w[1][b]);
                mma_f16(o[b][0], pf[0], pf[1], pf[2], pf[3], c0.x, c1.x);
                mma_f16(o[b][1], pf[0], pf[1], pf[2], pf[3], c0.y, c1.y);
                mma_f16(o[b][2], pf[0], pf[1], pf[2], pf[3], c0.z, c1.z);
                mma_f16(o[b][3], pf[0], pf[1], pf[2], pf[3], c0.w, c1.w);
            }
            ++taken;
            __syncwarp();                    // the chunk is read by all lanes before it is written again
            copy();
        }

        // Join the warps: row g's dims 32 b + 8 t .. + 7 of this lane, their reference and sum.
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        float* out = reinterpret_cast<float*>(smem + S::OUT);
        const bool any = work.g0 + warp < work.g1;
        if (any)
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float* to = out + (warp * ROWS + g) * S::OUT_STRIDE + 32 * b + 8 * t;
                *reinterpret_cast<float4*>(to) = make_float4(o[b][0][0] + o[b][0][2], o[b][1][0] + o[b][1][2], o[b][2][0] + o[b][2][2], o[b][3][0] + o[b][3][2]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(o[b][0][1] + o[b][0][3], o[b][1][1] + o[b][1][3], o[b][2][1] + o[b][2][3], o[b][3][1] + o[b][3][3]);
            }
        if (t == 0) stats[warp * ROWS + g] = make_float2(any && m != -INFINITY ? m + (float)(top_e - 8) : -INFINITY, l);
        __syncthreads();
        const bool complete = work.from == 0 && work.to == seq.cost;
        const int part = 2 * blockIdx.x + (work.from == 0 ? 1 : 0);
        float* part_rows = plan.rows + part * part_floats<B>();
        if (!complete && tid == 0) plan.parts[part] = {work.s, work.head, work.tile, work.from, work.to, seq.cost};
        for (int i = tid; i < ROWS * (S::DIM / 4); i += S::THREADS) {
            const int r = i / (S::DIM / 4), c = i % (S::DIM / 4) * 4;
            if (tile0 + r >= rows) break;                                          // r grows with i
            float ref = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) ref = larger(ref, stats[w * ROWS + r].x);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) {
                const float2 st = stats[w * ROWS + r];
                if (st.x == -INFINITY) continue;                                   // nothing was written there
                const float k = exp2f(st.x - ref);
                const float4 x = *reinterpret_cast<const float4*>(out + (w * ROWS + r) * S::OUT_STRIDE + c);
                sum = fmaf(k, st.y, sum);
                v.x = fmaf(k, x.x, v.x), v.y = fmaf(k, x.y, v.y), v.z = fmaf(k, x.z, v.z), v.w = fmaf(k, x.w, v.w);
            }
            if (complete) {
                const float inv = ref == -INFINITY ? 0.0f : 1.0f / sum;
                const int64_t at = (int64_t)(seq.q0 + (tile0 + r) / a.shared) * a.heads + work.head * a.shared + (tile0 + r) % a.shared;
                store4(a, at * S::DIM + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (c == 0 && a.lse) a.lse[at] = ref == -INFINITY ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
            } else {
                *reinterpret_cast<float4*>(part_rows + r * S::DIM + c) = v;
                if (c == 0) *reinterpret_cast<float2*>(part_rows + ROWS * S::DIM + 2 * r) = make_float2(ref, sum);
            }
        }
        __syncthreads();
    }
    if (dead) {
        // copies in flight must land before this CTA's shared memory is another's
        for (uint32_t i = taken; i < issued; ++i) mbar_wait_bounded(bars + (i % S::STAGES) * 8, (i / S::STAGES) & 1, a.limit_ns);
    }
}

// Joins the parts of the segments that were cut.  A segment's parts are a worker's last one (its
// start) and the first ones of the workers behind it; block (w, r) joins row r of the one that starts
// in worker w.
constexpr int JOIN_WARPS = 4;

template <int B>
__global__ void __launch_bounds__(JOIN_WARPS * 32) join_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    using S = Shape<B>;
    constexpr int VEC = S::DIM / 32;
    __shared__ float sums[JOIN_WARPS][S::DIM];
    __shared__ float2 stats[JOIN_WARPS];
    pdl_wait();
    const int w = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Part* parts = plan.parts;
    const int of = mx_ld(&parts[2 * w + 1].of), to0 = mx_ld(&parts[2 * w + 1].to);
    if (of < 0 || to0 >= of) return;                       // no segment starts here, or none that goes on
    const int s = mx_ld(&parts[2 * w + 1].seq), head = mx_ld(&parts[2 * w + 1].head), tile = mx_ld(&parts[2 * w + 1].tile);
    const Seq seq = seq_of(a, s, plan.whole);
    const int row = tile * ROWS + r;
    if (row >= seq.n * a.shared) return;
    // parts until the segment's end
    int n = 1;
    while (w + n < plan.workers && mx_ld(&parts[2 * (w + n)].of) >= 0 && mx_ld(&parts[2 * (w + n)].to) < of) ++n;
    n = min(n + 1, plan.workers - w);
    float ref = -INFINITY, sum = 0.0f, v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
    // the largest reference first: all of them in flight together
    for (int p = lane; p < n; p += 32) {
        const float* rows = plan.rows + (p == 0 ? 2 * w + 1 : 2 * (w + p)) * part_floats<B>();
        ref = larger(ref, mx_ld(rows + ROWS * S::DIM + 2 * r));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ref = larger(ref, __shfl_xor_sync(0xffffffffu, ref, d));
    for (int p = warp; p < n; p += JOIN_WARPS) {
        const float* rows = plan.rows + (p == 0 ? 2 * w + 1 : 2 * (w + p)) * part_floats<B>();
        const float k = share_of(mx_ld(rows + ROWS * S::DIM + 2 * r), ref);
        sum = fmaf(k, mx_ld(rows + ROWS * S::DIM + 2 * r + 1), sum);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = fmaf(k, mx_ld(rows + r * S::DIM + i * 32 + lane), v[i]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) sums[warp][i * 32 + lane] = v[i];
    if (lane == 0) stats[warp] = make_float2(ref, sum);
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < JOIN_WARPS; ++x) sum += stats[x].y;
    const float inv = ref == -INFINITY ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t)(seq.q0 + row / a.shared) * a.heads + head * a.shared + row % a.shared;
    for (int c = threadIdx.x * 4; c < S::DIM; c += JOIN_WARPS * 128) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < JOIN_WARPS; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(&sums[i][c]);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        store4(a, at * S::DIM + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
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

template <int B>
q4q_status run(const AttnArgs& a, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    using S = Shape<B>;
    const cudaError_t e = cudaFuncSetAttribute(attn_kernel<B>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e != cudaSuccess) return cudaGetLastError(), Q4Q_ERR_CUDA;
    Plan plan;
    plan.workers = info.sm_count;
    plan.least = S::WARPS;
    plan.whole = (a.max_pages << a.page_log) <= KV_GROUP * S::WARPS;
    plan.parts = static_cast<Part*>(workspace);
    plan.rows = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + mx_up((int64_t)sizeof(Part) * 2 * info.sm_count, 256));
    if (plan.whole) plan.least = 1;
    const q4q_status st = launch(attn_kernel<B>, dim3((unsigned)plan.workers), S::THREADS, S::BYTES, stream, a, plan);
    if (st != Q4Q_OK || plan.whole) return st;
    return launch(join_kernel<B>, dim3((unsigned)plan.workers, ROWS), JOIN_WARPS * 32, 0, stream, a, plan);
}

size_t workspace_bytes(int64_t head_dim, const DeviceInfo& info) {
    return (size_t)mx_up((int64_t)sizeof(Part) * 2 * info.sm_count, 256) + sizeof(float) * (size_t)(ROWS * head_dim + 2 * ROWS) * 2 * info.sm_count;
}

q4q_status check(AttnArgs& a, const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim,
                 const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages, int64_t max_pages, const int32_t* kv_len,
                 const int32_t* first, int64_t n_seqs, float scale, int causal, int64_t window, void* dst, float* lse, void* workspace,
                 size_t workspace_bytes_given, bool& empty, DeviceInfo& info) {
    q4q_status st = kv_check(n_pages, page_tokens, n_kv_heads, head_dim, a.page_log);
    if (st != Q4Q_OK) return st;
    if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % n_kv_heads || n_q < 0 || n_q >= (1 << 24) || n_seqs < 0 || n_seqs >= (1 << 20) ||
        max_pages < 0 || max_pages >= (1ll << 31) / page_tokens || window < 0)
        return Q4Q_ERR_SHAPE;
    if (q_stride < n_q_heads * head_dim || q_stride >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (!first && n_seqs > n_q) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(type) || !(scale == scale)) return Q4Q_ERR_ARG;
    empty = n_q == 0 || n_seqs == 0;
    if (empty) return Q4Q_OK;
    if (!q || !dst || !kv_len || !workspace || (max_pages > 0 && !pages) || (n_pages > 0 && !cache)) return Q4Q_ERR_NULL;
    const size_t size = mx_type_bytes(type);
    if (!aligned(q, size) || !aligned(dst, size) || !aligned(cache, 256) || !aligned(workspace, 256) || !aligned(pages, 4) || !aligned(kv_len, 4) ||
        !aligned(first, 4) || !aligned(lse, 4))
        return Q4Q_ERR_ALIGN;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    if (workspace_bytes_given < workspace_bytes(head_dim, info)) return Q4Q_ERR_WORKSPACE;
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache);
    a.pages = pages;
    a.kv_len = kv_len;
    a.first = first;
    a.n_q = n_q;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.window = window;
    a.n_seqs = (int)n_seqs;
    a.heads = n_q_heads;
    a.kv_heads = n_kv_heads;
    a.shared = n_q_heads / n_kv_heads;
    a.type = type;
    a.causal = causal != 0;
    a.align = aligned(q, 16) && aligned(dst, 16) && q_stride * size % 16 == 0 ? 16 : 1;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.dst = dst;
    a.lse = lse;
    a.limit_ns = WAIT_LIMIT_NS;
    a.fault = 0;
    return Q4Q_OK;
}

q4q_status dispatch(const AttnArgs& a, int64_t head_dim, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    switch (head_dim) {
        case 64: return run<2>(a, workspace, stream, info);
        case 96: return run<3>(a, workspace, stream, info);
        case 128: return run<4>(a, workspace, stream, info);
        default: return run<8>(a, workspace, stream, info);
    }
}

}  // namespace

unsigned int attn_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_attn_status, &z, sizeof(z));
    return v;
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_kv_attn_workspace_size(int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim, int64_t n_seqs, int type, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    if (!kv_dim_ok(head_dim) || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads || n_q < 0 || n_seqs < 0) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(type)) return Q4Q_ERR_ARG;
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    *bytes = workspace_bytes(head_dim, info);
    return Q4Q_OK;
}

extern "C" q4q_status q4q_kv_attn(const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads, int64_t head_dim,
                                  const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages, int64_t max_pages,
                                  const int32_t* kv_len, const int32_t* first, int64_t n_seqs, float scale, int causal, int64_t window,
                                  void* dst, float* lse, void* workspace, size_t workspace_bytes, q4q_stream_t stream) {
    AttnArgs a{};
    DeviceInfo info;
    bool empty;
    const q4q_status st = check(a, q, q_stride, type, n_q, n_q_heads, n_kv_heads, head_dim, cache, n_pages, page_tokens, pages, max_pages, kv_len,
                                first, n_seqs, scale, causal, window, dst, lse, workspace, workspace_bytes, empty, info);
    if (st != Q4Q_OK || empty) return st;
    return dispatch(a, head_dim, workspace, (cudaStream_t)stream, info);
}

extern "C" q4q_status q4q_debug_kv_attn_timeout(const void* q, int64_t q_stride, int type, int64_t n_q, int n_q_heads, int n_kv_heads,
                                                int64_t head_dim, const void* cache, int64_t n_pages, int page_tokens, const int32_t* pages,
                                                int64_t max_pages, const int32_t* kv_len, int64_t n_seqs, float scale, void* dst,
                                                void* workspace, size_t workspace_bytes, uint64_t limit_ns, q4q_stream_t stream) {
    if (limit_ns < 1 || limit_ns > WAIT_LIMIT_NS) return Q4Q_ERR_ARG;
    AttnArgs a{};
    DeviceInfo info;
    bool empty;
    const q4q_status st = check(a, q, q_stride, type, n_q, n_q_heads, n_kv_heads, head_dim, cache, n_pages, page_tokens, pages, max_pages, kv_len,
                                nullptr, n_seqs, scale, 1, 0, dst, nullptr, workspace, workspace_bytes, empty, info);
    if (st != Q4Q_OK || empty) return st;
    a.limit_ns = limit_ns;
    a.fault = 1;
    return dispatch(a, head_dim, workspace, (cudaStream_t)stream, info);
}
