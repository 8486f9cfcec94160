// q4q_attn_tc.cu -- attention over the paged 4-bit cache on the tcgen05 tensor cores: prompts and chunks of
// them, bf16 and fp16, heads of 64, 96 and 128 values.
//
// The mathematics is that of q4q_attn_kernel.cuh; here many rows of queries share a key, so keys and values are
// decoded once, and both products are 128 x 128 MMAs of fp16 with fp32 sums in tensor memory.  Keys are two operands that add up to (code - 8) d
// exactly: as one, rounded to fp16 (2^-12), they moved the weights by that much of a score: bf16 rows whose scores spread over 6 nats were
// 1.91e-3 from 64 bits (512 rows over 8192 keys), now 1.66e-3, of which
// their results' own rounding is 1.64e-3.  The second product costs 96.6 -> 103 us there, 540 -> 587 for 8 such sequences.  Values are
// (code - 8) d in fp16 (one rounding, 2^-12 at most; d is at most 8188, so all are finite).  Queries become fp16 of a power of
// two times their row, its largest in [2^14, 2^15) (exact down to 2^-28 of that: below, multiples of 2^-39 of it), weights are rounded to fp16:
// values and weights are 2^3 below a bf16 result's own rounding, and as large as an fp16 result's.  The weight of the maximum that a row
// refers to is 2^7, and the reference moves only when a maximum passes it by 2^8, so the largest weight is between 2^7 and fp16's
// range, and weights down to 2^-21 of it are normal numbers, others multiples of 2^-31 of it.  (With a weight of 1 those of 2^-14 were the last:
// where a first key without a value outweighs 499 others by 2^20, bf16 results of the others were 1.7e-2 from 64 bits.)
//
// A CTA takes 256 rows (tokens x shared heads of a key-value head) as two tiles of 128 rows against steps of 128 keys:
//   warps 0-3, 4-7   softmax of a tile, a thread a row: S from tensor memory twice (maximum, then weights), P over S,
//                    the sums' rescaling, the result
//   warps 8-15       decode chunks to the MMAs' operands: K [keys][dims], V^T [dims][keys], 128-byte swizzle, two stages
//                    each.  Codes and scales come straight from the cache into registers, a step ahead.  A lane of K holds 8
//                    dims of a key, a 16-byte unit (dims of a unit in the nibbles' order 0 4 1 5 2 6 3 7, queries alike); V's
//                    words hold two keys of 4 dims, which is what a lane of stmatrix holds of an 8 x 8 matrix [dim][key], so
//                    rows of V^T are dims 4 g + n at place 8 n + g of their block, and results are put back in order from
//                    registers
//   warp 16          MMAs: S_i = Q_i K^T, O_i += P_i V, the two tiles in turn, so that one's softmax runs beside the
//                    other's MMAs
//   warps 17-19      the next piece's queries
// Steps of all pieces (sequence, head, 256 rows) in a row are cut into equal shares, one a CTA and SM; parts of a
// piece are joined by a second kernel in order.
//
// Measured in a graph (heads 32/8 of 128): bf16, 512 rows behind 7680 keys 103 us (647 TFLOP/s), 8 such sequences 580 us (918
// TFLOP/s), two prompts of 2048 with a window of 1024 135 us; fp16 103 and 137 us.  A row's 128 scores are read twice, exponentiated
// and written back by one thread, and only the other tile's MMAs run beside that; the forms spill (276 to 288 bytes of stores, 396 to 404
// of loads); a piece's start and end cost about 10 us each time, the shares 4.4 us.
#include "q4q_attn_kernel.cuh"

namespace q4q {
namespace {

constexpr int TC_TILE = 128;             // rows of a tile and keys of a step
constexpr int TC_ROWS = 2 * TC_TILE;     // rows of a piece
constexpr int TC_CHUNKS = TC_TILE / KV_GROUP;
constexpr int TC_DECODERS = TC_CHUNKS;   // warps, one for each chunk of a step
constexpr int TC_ISSUER = 8 + TC_DECODERS;
constexpr int TC_LOADERS = 3;
constexpr int TC_THREADS = (TC_ISSUER + 1 + TC_LOADERS) * 32;
// Registers a thread: at launch, and as the warpgroups share them out, in all the same number.
constexpr int TC_REGS = 96, TC_SOFTMAX_REGS = 128, TC_DECODE_REGS = 80, TC_OTHER_REGS = 64;
static_assert(256 * TC_SOFTMAX_REGS + 256 * TC_DECODE_REGS + 128 * TC_OTHER_REGS <= TC_THREADS * TC_REGS, "registers of the launch");
constexpr int TC_SNAP = 3;               // steps that a share may be longer or shorter, so that it ends with a piece
constexpr float TC_TOP = 7.0f, TC_LAG = 8.0f;   // log2 of the weight of the maximum referred to; how far a maximum may pass it
constexpr int TC_INFOS = 4;              // steps whose notes are kept: decoders are at most 2 ahead of the softmax

template <int B_, typename T_>
struct Tc {
    using T = T_;                                                  // of queries and results
    static constexpr int B = B_, DIM = 32 * B;
    static constexpr int ATOMS = (B + 1) / 2;                      // of 64 dims
    static constexpr int Q_BYTES = ATOMS * TC_TILE * 128, V_BYTES = 2 * DIM * 128;
    static constexpr int STAGES = 2;
    // Keys as two operands, (code - 8) times the scale's upper 7 bits and its other 4; where two stages of both do not fit
    // (heads of 96 and 128), one.
    static constexpr int K_STAGES = B <= 2 ? 2 : 1, K_BYTES = 2 * Q_BYTES;
    // barriers
    enum { K_FULL = 0, K_EMPTY = K_FULL + STAGES, V_FULL = K_EMPTY + STAGES, V_EMPTY = V_FULL + STAGES, Q_FIRST = V_EMPTY + STAGES, Q_FULL, Q_FREE, S_FULL,
           P_FULL = S_FULL + 2, O_DONE = P_FULL + 2, DRAIN = O_DONE + 2, BARS };
    static constexpr int STOP = BARS * 8, TMEM = STOP + 4;
    static constexpr int WORDS = (TMEM + 4 + 7) / 8 * 8;           // scan and broadcast words
    static constexpr int GONE = 512, ODD = GONE + TC_INFOS * 8;    // [TC_INFOS][8] bytes: chunks that are not there; with scales that are no number
    static constexpr int WHICH = 1024;                             // [TC_INFOS][128] bytes: bit b, the key's scale of V's block b is no number
    static constexpr int SCALE = 1536;                             // [2][256] fp32: what a row's scores are multiplied by, of a piece and the next
    static constexpr int Q = 4096;
    static constexpr int K = Q + 2 * Q_BYTES, V = K + K_STAGES * K_BYTES;
    static constexpr int BYTES = V + STAGES * V_BYTES + 1024;      // the tiles start on 1024 bytes
    static_assert(WORDS + (TC_THREADS / 32 + 7) * 8 <= GONE && ODD + TC_INFOS * 8 <= WHICH, "small things before the tiles");
    static_assert(K % 1024 == 0 && V % 1024 == 0 && BYTES <= 227 * 1024, "shared memory");
};

// ------------------------------------------------------------ the steps --

// The steps of a tile pair: c0 the first, and how many it is counted as (at least one, so that a piece that sees no key
// is written too).
__device__ __forceinline__ int tc_cost(const AttnArgs& a, const Seq& s, int tile, int& c0, int& c1) {
    int lo, hi, unused;
    keys_of(a, s, tile * TC_ROWS, lo, unused);
    keys_of(a, s, min(tile * TC_ROWS + TC_ROWS, s.n * a.shared) - 1, unused, hi);
    c0 = lo / TC_TILE;
    c1 = (hi + TC_TILE - 1) / TC_TILE;
    return max(1, c1 - c0);
}

// Steps of all tiles of a head.  team 1: this thread alone; 32: the lanes of the warp together.
__device__ __forceinline__ int64_t tc_head_cost(const AttnArgs& a, const Seq& s, int team) {
    int64_t sum = 0;
    int c0, c1;
    for (int t = (threadIdx.x & 31) % team; t < s.tiles; t += team) sum += tc_cost(a, s, t, c0, c1);
    if (team > 1)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// The tile that step `rel` of a head lies in, its steps; rel from its start.
__device__ __forceinline__ int tc_tile_of(const AttnArgs& a, const Seq& s, int64_t& rel, int& cost, int team) {
    int c0, c1;
    if (team == 1) {
        for (int tile = 0;; ++tile) {
            cost = tc_cost(a, s, tile, c0, c1);
            if (rel < cost || tile + 1 >= s.tiles) return tile;
            rel -= cost;
        }
    }
    const int lane = threadIdx.x & 31;
    for (int t0 = 0;; t0 += 32) {
        const int mine = t0 + lane < s.tiles ? tc_cost(a, s, t0 + lane, c0, c1) : 0;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const uint32_t behind = __ballot_sync(0xffffffffu, inc > rel);
        if (behind || t0 + 32 >= s.tiles) {
            const int at = behind ? __ffs(behind) - 1 : min(31, s.tiles - 1 - t0);
            cost = __shfl_sync(0xffffffffu, mine, at);
            rel -= __shfl_sync(0xffffffffu, inc, at) - cost;
            return t0 + at;
        }
        rel -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

// A walk over a worker's steps: pieces, one after another.
struct TcWalk {
    int64_t left;              // steps behind the piece
    int s, head, tile, from;   // where they start
    Seq seq;
    // the piece: steps g0 .. g1 - 1 of the sequence, `first` .. `last` - 1 of the `of` that its tile is counted as
    int p_s, p_head, p_tile, first, last, of, g0, g1;
    Seq p_seq;
    bool valid;
};

__device__ __forceinline__ void tc_next(const AttnArgs& a, TcWalk& w) {
    w.valid = false;
    while (w.left > 0) {
        if (w.tile >= w.seq.tiles || w.head >= a.kv_heads) {
            w.from = 0;
            w.tile = 0;
            if (w.seq.tiles == 0 || ++w.head >= a.kv_heads) {
                w.head = 0;
                w.seq = seq_of<TC_ROWS>(a, ++w.s, false);
            }
            continue;
        }
        int c0, c1;
        const int cost = tc_cost(a, w.seq, w.tile, c0, c1);
        if (w.from >= cost) {                        // a share that starts with the next piece
            w.from = 0;
            ++w.tile;
            continue;
        }
        w.p_s = w.s;
        w.p_head = w.head;
        w.p_tile = w.tile;
        w.p_seq = w.seq;
        w.first = w.from;
        w.last = (int)min((int64_t)cost, w.from + w.left);
        w.of = cost;
        w.g0 = min(c0 + w.first, c1);
        w.g1 = min(c0 + w.last, c1);
        w.left -= w.last - w.first;
        if (w.last == cost) {
            w.from = 0;
            ++w.tile;
        } else {
            w.from = w.last;
        }
        w.valid = true;
        return;
    }
}

// This worker's share of all steps: its walk.  Few sequences: each warp takes a run of them, its lanes their tiles; many: each
// thread a run.  words: TC_THREADS / 32 + 7 words of shared memory.
__device__ __forceinline__ TcWalk tc_share(const AttnArgs& a, const Plan& plan, int64_t* words) {
    constexpr int WARPS = TC_THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = a.n_seqs <= 8 * WARPS ? 32 : 1, runs = TC_THREADS / team, run = tid / team;
    const int per = (a.n_seqs + runs - 1) / runs, s0 = min(run * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
    int64_t sum = 0;
    for (int s = s0; s < s1; ++s) sum += a.kv_heads * tc_head_cost(a, seq_of<TC_ROWS>(a, s, false), team);
    int64_t inc = sum;
    if (team == 1)
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
    const bool works = blockIdx.x < workers;
    // A share ends with a piece where one ends near: what is cut has to be joined.
    const int64_t snap = min(total / workers / 6, (int64_t)TC_SNAP);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t u = works ? (total * (blockIdx.x + k) + workers - 1) / workers : total;
        if (u >= total && tid == 0) words[WARPS + 1 + k] = total;
        if (u < total && before <= u && u < before + sum) {
            int s = s0, cost;
            int64_t head_cost, base = before;
            while (true) {
                head_cost = tc_head_cost(a, seq_of<TC_ROWS>(a, s, false), team);
                if (u < base + head_cost * a.kv_heads) break;
                base += head_cost * a.kv_heads;
                ++s;
            }
            const Seq seq = seq_of<TC_ROWS>(a, s, false);
            int64_t rel = u - base;
            const int64_t head = rel / head_cost;
            rel -= head * head_cost;
            const int tile = tc_tile_of(a, seq, rel, cost, team);
            // to the piece's end, which the walk finds by itself, or to its start
            const int64_t move = rel == 0 ? 0 : cost - rel <= snap ? cost - rel : rel <= snap ? -rel : 0;
            words[WARPS + 1 + k] = u + move;
            if (k == 0) {
                words[WARPS + 3] = s;
                words[WARPS + 4] = head;
                words[WARPS + 5] = tile;
                words[WARPS + 6] = rel + move;
            }
        }
    }
    __syncthreads();
    TcWalk w;
    w.left = words[WARPS + 2] - words[WARPS + 1];
    w.valid = false;
    if (w.left <= 0) return w;
    w.s = (int)words[WARPS + 3];
    w.head = (int)words[WARPS + 4];
    w.tile = (int)words[WARPS + 5];
    w.from = (int)words[WARPS + 6];
    w.seq = seq_of<TC_ROWS>(a, w.s, false);
    return w;
}

// What every role's waits look at.
struct TcWaits {
    uint32_t bars;
    volatile int* stop;
    uint64_t limit_ns;
    // false: the wait ran out, here or elsewhere in the CTA (the whole warp calls it)
    __device__ __forceinline__ bool operator()(int bar, uint32_t parity) const {
        const uint32_t at = bars + bar * 8;
        const bool ok = mbar_try_wait(at, parity) || mbar_wait_until(at, parity, stop, limit_ns);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (!*stop && (threadIdx.x & 31) == 0) record_error(&g_attn_status, DEV_TIMEOUT);
        __syncwarp();
        *stop = 1;
        return false;
    }
    __device__ __forceinline__ void arrive(int bar) const { mbar_arrive(bars + bar * 8); }
};

// ------------------------------------------------------------- the roles --

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// WORDS words of the cache
template <int WORDS>
__device__ __forceinline__ void ldg(const uint8_t* p, uint32_t (&v)[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 x = mx_ld(reinterpret_cast<const uint4*>(p) + i);
            v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
    } else if constexpr (WORDS == 2) {
        asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) v[i] = mx_ld(reinterpret_cast<const uint32_t*>(p) + i);
    }
}

// B scales of a token, two a word
template <int B>
__device__ __forceinline__ void ldg_scales(const uint8_t* p, uint32_t (&v)[(B + 1) / 2]) {
    if constexpr (B % 2 == 0) {
        ldg<B / 2>(p, v);
    } else {
        uint32_t h[B + 1];
#pragma unroll
        for (int i = 0; i < B; ++i) h[i] = mx_ld(reinterpret_cast<const uint16_t*>(p) + i);
        h[B] = 0;
#pragma unroll
        for (int i = 0; i < (B + 1) / 2; ++i) v[i] = h[2 * i] | h[2 * i + 1] << 16;
    }
}

// Decoders: warp d takes chunk d of a step; its keys first, so that the step's scores can start.
template <typename C>
__device__ __forceinline__ void tc_decode(const AttnArgs& a, TcWalk w, const TcWaits& wait, uint32_t base, uint8_t* smem) {
    constexpr int B = C::B, W = (B + 1) / 2;
    const int lane = threadIdx.x & 31, d = (threadIdx.x >> 5) - 8, in_page = a.page_log - 4;
    // K: lanes of a quarter-warp take 8 dims of keys i and i + 4 of an octet, whose 16-byte units then differ; V: two keys of
    // 4 dims of each block
    const int i = (lane >> 3) + ((lane >> 2) & 1) * 4, t = lane & 3;
    // The walk is two steps ahead of the decoding: `next` is the step whose chunks' pages are being looked up, `here` the one
    // whose codes are on their way.
    struct Step {
        int g, len, head;
        int page;                                    // as looked up, not looked at before the codes are loaded
        const uint8_t* chunk;                        // null: not there
        bool any;
    } next, here;
    next.any = false;
    int g = 0;
    tc_next(a, w);
    if (w.valid) g = w.g0;
    const auto find = [&]() {
        while (w.valid && g >= w.g1) {
            tc_next(a, w);
            if (w.valid) g = w.g0;
        }
        next.any = w.valid;
        if (!w.valid) return;
        next.g = g;
        next.len = w.p_seq.len;
        next.head = w.p_head;
        next.page = -1;
        const int group = g * TC_CHUNKS + d;
        if (group * KV_GROUP < next.len) next.page = mx_ld(a.pages + w.p_s * a.max_pages + (group >> in_page));
        ++g;
    };
    uint32_t kx[2][B], ks[2][W], vx[2][B], vs[2][2][W];
    const auto load_k = [&](Step& s) {
        s.chunk = nullptr;
        if (!s.any || s.page < 0 || s.page >= a.n_pages) return;
        s.chunk = a.cache + kv_chunk_offset(s.page, s.head, (s.g * TC_CHUNKS + d) & ((1 << in_page) - 1), a.kv_heads, a.page_log, C::DIM);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ldg<B>(s.chunk + ((8 * j + i) * 4 + t) * 4 * B, kx[j]);
            ldg_scales<B>(s.chunk + 16 * C::DIM + (8 * j + i) * 2 * B, ks[j]);
        }
    };
    const auto load_v = [&](const Step& s) {
        if (!s.chunk) return;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ldg<B>(s.chunk + 8 * C::DIM + (j * 32 + lane) * 4 * B, vx[j]);
#pragma unroll
            for (int k = 0; k < 2; ++k) ldg_scales<B>(s.chunk + 17 * C::DIM + (8 * j + 2 * t + k) * 2 * B, vs[j][k]);
        }
    };
#pragma unroll
    for (int x = 0; x < 2 * B; ++x) kx[x / B][x % B] = vx[x / B][x % B] = 0u;
#pragma unroll
    for (int x = 0; x < 2 * W; ++x) ks[x / W][x % W] = vs[x / W][0][x % W] = vs[x / W][1][x % W] = 0u;
    find();
    here = next;
    load_k(here);
    load_v(here);
    find();
    for (uint32_t steps = 0; here.any; ++steps) {
        const uint32_t stage = steps % C::STAGES, round = steps / C::STAGES, note = steps % TC_INFOS;
        const uint32_t k_stage = steps % C::K_STAGES, k_round = steps / C::K_STAGES;
        const int key0 = here.g * TC_TILE + d * KV_GROUP, left = here.len - key0;     // of the chunk; its tokens
        const bool gone = !here.chunk;
        here = next;
        if (lane == 0) {
            smem[C::GONE + note * TC_CHUNKS + d] = gone;
            if (gone && left > 0) record_error(&g_attn_status, Q4Q_ERR_ARG);
        }
        if (k_round > 0 && !wait(C::K_EMPTY + k_stage, (k_round - 1) & 1)) return;
        {
            const uint32_t to = base + C::K + k_stage * C::K_BYTES + (d * KV_GROUP + i) * 128;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const uint32_t s2 = __byte_perm(ks[j][b / 2], 0, b % 2 ? 0x3232 : 0x1010);
                    const uint4 v = nibbles_to_f16x8(kx[j][b]);
                    const uint32_t at = to + (b / 2) * TC_TILE * 128 + j * 1024 + ((((b % 2) * 4 + t) ^ i) << 4);
                    const uint32_t high = s2 & 0xFFF0FFF0u;
                    sts128(at, half2_mul(v.x, high), half2_mul(v.y, high), half2_mul(v.z, high), half2_mul(v.w, high));
                    const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&s2), *reinterpret_cast<const __half2*>(&high));
                    const uint32_t low = *reinterpret_cast<const uint32_t*>(&rest);
                    sts128(at + C::Q_BYTES, half2_mul(v.x, low), half2_mul(v.y, low), half2_mul(v.z, low), half2_mul(v.w, low));
                }
        }
        fence_async();
        __syncwarp();
        if (lane == 0 && !(a.fault && blockIdx.x == 0 && d == 0 && steps == 0)) wait.arrive(C::K_FULL + k_stage);
        load_k(here);
        // Scales of keys that are not there become 0, and so do those that are no number: the softmax marks the rows that see
        // those.
        if (gone || left < KV_GROUP)
#pragma unroll
            for (int x = 0; x < 4 * W; ++x)
                if (gone || x / (2 * W) * 8 + 2 * t + x / W % 2 >= left) vs[x / (2 * W)][x / W % 2][x % W] = 0u;
        uint32_t no = 0;
#pragma unroll
        for (int x = 0; x < 4 * W; ++x) no |= __vcmpgtu2(vs[x / (2 * W)][x / W % 2][x % W] & 0x7FFF7FFFu, 0x7BFF7BFFu);
        const bool odd = __any_sync(0xffffffffu, no != 0);
        if (lane == 0) smem[C::ODD + note * TC_CHUNKS + d] = odd;
        if (odd) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = x / 2, k = x % 2;
                uint32_t which = 0;
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    const uint32_t bad = __vcmpgtu2(vs[j][k][q] & 0x7FFF7FFFu, 0x7BFF7BFFu);
                    which |= (bad & 1u ? 1u << (2 * q) : 0u) | (bad >> 16 ? 2u << (2 * q) : 0u);
                    vs[j][k][q] &= ~bad;
                }
                if (lane < 4) smem[C::WHICH + note * TC_TILE + d * KV_GROUP + 8 * j + 2 * t + k] = (uint8_t)which;
            }
        }
        if (round > 0 && !wait(C::V_EMPTY + stage, (round - 1) & 1)) return;
        {
            // matrices of 8 dims x 8 keys, row g of matrix n at place 32 b + 8 n + g; the address that this lane gives is that of
            // row lane % 8 of matrix lane / 8
            const uint32_t to = base + C::V + stage * C::V_BYTES + (d >> 2) * C::DIM * 128 + lane * 128;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const uint32_t s2 = __byte_perm(vs[j][0][b / 2], vs[j][1][b / 2], b % 2 ? 0x7632 : 0x5410);
                    const uint4 v = nibbles_to_f16x8(vx[j][b]);
                    stmatrix4(to + b * 32 * 128 + ((((2 * d + j) & 7) ^ (lane & 7)) << 4), half2_mul(v.x, s2), half2_mul(v.y, s2), half2_mul(v.z, s2),
                              half2_mul(v.w, s2));
                }
        }
        load_v(here);
        fence_async();
        __syncwarp();
        if (lane == 0) wait.arrive(C::V_FULL + stage);
        find();
    }
}

// A = P [128 rows x 16 keys] from tensor memory, or queries from shared memory; B from shared memory, K-major.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// fp32 sums, fp16 operands, both K-major, N columns
__host__ __device__ constexpr uint32_t tc_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TC_TILE >> 4) << 24); }

// tensor memory: S and P of tile i at 128 i, O at 256 + 128 i
template <typename C>
__device__ __forceinline__ void tc_issue(const AttnArgs& a, TcWalk w, const TcWaits& wait, uint32_t base, uint32_t tmem) {
    const bool one = elect_one();
    uint32_t steps = 0, pieces = 0;
    bool ok = true;
    const auto commit = [&](int bar) {
        if (one) mma_commit(wait.bars + bar * 8);
    };
    const auto scores = [&](int i, uint32_t stage) {
        const uint64_t q = desc_sw128(base + C::Q + i * C::Q_BYTES), k = desc_sw128(base + C::K + stage * C::K_BYTES);
        if (one)
#pragma unroll
            for (int x = 0; x < 4 * C::B; ++x) {
                const uint64_t at = ((x % (2 * C::B) / 4) * TC_TILE * 128 + (x % (2 * C::B) % 4) * 32) >> 4;
                tc_mma_ss(tmem + i * TC_TILE, q + at, k + at + (x / (2 * C::B)) * (C::Q_BYTES >> 4), tc_idesc(TC_TILE), x > 0);
            }
        __syncwarp();
    };
    const auto values = [&](int i, uint32_t stage, bool more) {
        const uint64_t v = desc_sw128(base + C::V + stage * C::V_BYTES);
        if (one)
#pragma unroll
            for (int x = 0; x < TC_TILE / 16; ++x)
                tc_mma_ts(tmem + 2 * TC_TILE + i * TC_TILE, tmem + i * TC_TILE + x * 8, v + (((x / 4) * C::DIM * 128 + (x % 4) * 32) >> 4),
                          tc_idesc(C::DIM), more || x > 0);
        __syncwarp();
    };
    while (ok) {
        tc_next(a, w);
        if (!w.valid) break;
        const int n = w.g1 - w.g0;
        if (n <= 0) continue;
        // the first step's scores
        ok = (pieces == 0 ? wait(C::Q_FIRST, 0) : wait(C::Q_FULL, (pieces - 1) & 1)) &&
             wait(C::K_FULL + steps % C::K_STAGES, (steps / C::K_STAGES) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            scores(i, steps % C::K_STAGES);
            commit(C::S_FULL + i);
        }
        commit(C::K_EMPTY + steps % C::K_STAGES);
        if (n == 1) commit(C::Q_FREE);
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t at = steps + j, stage = at % C::STAGES, parity = (at / C::STAGES) & 1, next = (at + 1) % C::K_STAGES;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ok = ok && wait(C::P_FULL + i, at & 1) && (i > 0 || wait(C::V_FULL + stage, parity));
                if (!ok) break;
                tc_fence_after();
                values(i, stage, j > 0);
                if (j + 1 == n) {
                    commit(C::O_DONE + i);
                } else {
                    // behind the product that reads P: MMAs run in the order they were issued in
                    if (i == 0) ok = wait(C::K_FULL + next, ((at + 1) / C::K_STAGES) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    scores(i, next);
                    commit(C::S_FULL + i);
                }
            }
            if (!ok) break;
            commit(C::V_EMPTY + stage);
            if (j + 1 < n) commit(C::K_EMPTY + next);
            if (j + 2 == n) commit(C::Q_FREE);
        }
        steps += n;
        ++pieces;
    }
    // nothing is in flight when tensor and shared memory are given back
    commit(C::DRAIN);
    mbar_wait_bounded(wait.bars + C::DRAIN * 8, 0, a.limit_ns);
    __syncwarp();
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
          "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Loads issued so far are done; that the registers go through it keeps their uses behind it.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                   "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                   "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                   "+r"(r[31])::"memory");
}

template <typename C, typename F>
__device__ __forceinline__ void tc_rows(const AttnArgs& a, const TcWalk& w, int warp, int warps, uint32_t parity, uint32_t base, uint8_t* smem, F ready);

// Two results in 16 bits each.  fp16: weights rounded up on their own may lift a mean of values of 65504 past its range.
__device__ __forceinline__ float tc_limited(float x) { return x > 65504.0f ? 65504.0f : x < -65504.0f ? -65504.0f : x; }
template <typename T>
__device__ __forceinline__ uint32_t tc_bits(float x, float y) {
    if constexpr (std::is_same_v<T, __half>) {
        return half2_bits(tc_limited(x), tc_limited(y));
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// The softmax of tile i, a thread a row: queries, weights, and at a piece's end the results.
template <typename C>
__device__ __forceinline__ void tc_softmax(const AttnArgs& a, const Plan& plan, TcWalk w, const TcWaits& wait, uint32_t base, uint8_t* smem, uint32_t tmem) {
    constexpr int B = C::B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;                       // this warp's 32 lanes of tensor memory
    const uint32_t s_at = tmem + lanes + i * TC_TILE, o_at = tmem + lanes + 2 * TC_TILE + i * TC_TILE;
    uint32_t steps = 0, pieces = 0;
    while (true) {
        tc_next(a, w);
        if (!w.valid) return;
        const Seq& seq = w.p_seq;
        const int rows = seq.n * a.shared, at_row = w.p_tile * TC_ROWS + i * TC_TILE + r, row = min(at_row, rows - 1), n = w.g1 - w.g0;
        const int64_t at = (int64_t)(seq.q0 + row / a.shared), head = w.p_head * a.shared + row % a.shared;
        int lo, hi;
        keys_of(a, seq, row, lo, hi);
        const int lo_all = __reduce_max_sync(0xffffffffu, lo), hi_all = __reduce_min_sync(0xffffffffu, hi);
        float scale = 0.0f, ref = NONE, l = 0.0f;                            // weights are exp2(score - ref)
        uint32_t poison = 0;                                                  // blocks in which the row sees a value that is no number
        // Blocks of values that are no number, of keys of a step that this row sees.  The step's values are decoded by the time of
        // the next step's scores, or of the result.
        const auto marks = [&](uint32_t step, int key0) {
            const uint64_t odd = *reinterpret_cast<volatile uint64_t*>(smem + C::ODD + (step % TC_INFOS) * TC_CHUNKS);
            if (!odd) return;
            for (int k = max(lo - key0, 0); k < min(hi - key0, TC_TILE); ++k)
                if ((odd >> (k / 16 * 8)) & 1) poison |= *reinterpret_cast<volatile uint8_t*>(smem + C::WHICH + (step % TC_INFOS) * TC_TILE + k);
        };
        if (n > 0 && pieces == 0) {
            tc_rows<C>(a, w, warp, 8, 0, base, smem, [] {});
            if (lane == 0) wait.arrive(C::Q_FIRST);
        }
        for (int j = 0; j < n; ++j, ++steps) {
            if (!wait(C::S_FULL + i, steps & 1)) return;
            tc_fence_after();
            if (j == 0) scale = *reinterpret_cast<volatile float*>(smem + C::SCALE + ((pieces & 1) * TC_ROWS + i * TC_TILE + r) * 4);
            const int key0 = (w.g0 + j) * TC_TILE;
            const uint64_t gone = *reinterpret_cast<volatile uint64_t*>(smem + C::GONE + (steps % TC_INFOS) * TC_CHUNKS);
            const bool edge = key0 < lo_all || key0 + TC_TILE > hi_all || gone != 0;
            if (j > 0) marks(steps - 1, key0 - TC_TILE);
            // keys of this step that the row sees: from .. to - 1, but for chunks that are not there
            const int from = max(lo - key0, 0), to = min(hi - key0, TC_TILE);
            uint32_t seen[4];                        // bit k % 32 of seen[k / 32]: the row sees key k of the step
            if (edge)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int f = min(max(from - 32 * q, 0), 32), t = min(max(to - 32 * q, 0), 32);
                    seen[q] = t > f ? (0xffffffffu >> (32 - (t - f))) << f : 0u;
                    if ((gone >> (16 * q)) & 1) seen[q] &= 0xffff0000u;
                    if ((gone >> (16 * q + 8)) & 1) seen[q] &= 0x0000ffffu;
                }
            // The row's maximum, the last columns first: the first ones are still in registers when the weights begin with them.
            // (Reading halves of the columns once, with a maximum for each, came out slower: 621 us against 539 for 8 x 512 rows
            // over 8192 keys.)
            uint32_t x[2][32];
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const auto maximum = [&](auto of_edge) {
                tmem_ld32(s_at + 96, x[1]);
                tmem_ld_done(x[1]);
#pragma unroll
                for (int q = 3; q >= 0; --q) {
                    uint32_t(&v)[32] = x[q & 1];
                    if (q > 0) tmem_ld32(s_at + 32 * (q - 1), x[(q - 1) & 1]);
                    if constexpr (decltype(of_edge)::value) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) top[k & 3] = (seen[q] >> k) & 1 ? fmaxf(top[k & 3], __uint_as_float(v[k])) : top[k & 3];
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
#pragma unroll
                            for (int n = 0; n < 4; ++n) top[n] = fmaxf(top[n], fmaxf(__uint_as_float(v[k + 2 * n]), __uint_as_float(v[k + 2 * n + 1])));
                    }
                    if (q > 0) tmem_ld_done(x[(q - 1) & 1]);
                }
            };
            if (edge) maximum(std::true_type{});
            else maximum(std::false_type{});
            const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            const float y = most == -INFINITY ? -INFINITY : most * scale;
            if (__any_sync(0xffffffffu, y > ref + (TC_TOP + TC_LAG))) {
                const float to_ref = y > ref + (TC_TOP + TC_LAG) ? y - TC_TOP : ref, down = exp2f(ref - to_ref);
                ref = to_ref;
                l *= down;
                // this step's scores are there, so the products issued before them are done with the sums
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < C::DIM; c += 16) {
                        uint32_t old[16];
                        tmem_ld<16>(o_at + c, old);
#pragma unroll
                        for (int k = 0; k < 16; ++k) old[k] = __float_as_uint(__uint_as_float(old[k]) * down);
                        tmem_st16(o_at + c, old);
                    }
                }
            }
            uint64_t sum[2] = {0, 0};
            const uint64_t scale2 = pack2(scale, scale), ref2 = pack2(-ref, -ref);
            const auto weights = [&](auto of_edge) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t(&v)[32] = x[q & 1];
                    if (q < 3) tmem_ld32(s_at + 32 * (q + 1), x[(q + 1) & 1]);
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float z0, z1;
                        unpack2(ffma2(pair_of(v[2 * k], v[2 * k + 1]), scale2, ref2), z0, z1);
                        z0 = ex2(z0);
                        z1 = ex2(z1);
                        if constexpr (decltype(of_edge)::value) {
                            z0 = (seen[q] >> (2 * k)) & 1 ? z0 : 0.0f;
                            z1 = (seen[q] >> (2 * k + 1)) & 1 ? z1 : 0.0f;
                        }
                        sum[k & 1] = fadd2(sum[k & 1], pack2(z0, z1));
                        p[k] = half2_bits(z0, z1);
                    }
                    if (q < 3) tmem_ld_done(x[(q + 1) & 1]);
                    tmem_st16(s_at + 16 * q, p);                              // over scores that have been read
                }
            };
            if (edge) weights(std::true_type{});
            else weights(std::false_type{});
            float l0, l1;
            unpack2(fadd2(sum[0], sum[1]), l0, l1);
            l += l0 + l1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) wait.arrive(C::P_FULL + i);
        }
        // the results
        if (n > 0) {
            if (!wait(C::O_DONE + i, pieces & 1)) return;
            tc_fence_after();
            ++pieces;
            marks(steps - 1, (w.g1 - 1) * TC_TILE);
        }
        const bool complete = w.first == 0 && w.last == w.of, there = at_row < rows;
        const int part = 2 * blockIdx.x + (w.first == 0 ? 1 : 0);
        float* part_row = plan.rows + (int64_t)part * (TC_ROWS * (C::DIM + 2)) + (i * TC_TILE + r) * C::DIM;
        if (!complete && tid == 0) plan.parts[part] = {w.p_s, w.p_head, w.p_tile, w.first, w.last, w.of};
        const bool none = ref == NONE && l == 0.0f;                           // scores that are all NaN leave a NaN in l
        const float inv = complete ? (none ? 0.0f : 1.0f / l) : 1.0f;
        typename C::T* out = static_cast<typename C::T*>(a.dst) + (at * a.heads + head) * C::DIM;
#pragma unroll 1
        for (int b = 0; b < B; ++b) {
            uint32_t x[32];
            if (n > 0) tmem_ld<32>(o_at + 32 * b, x);
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                // place 8 n + g of the block is dim 4 g + n
                const float o = n > 0 && !none ? __uint_as_float(x[k]) * inv : 0.0f;
                v[4 * (k % 8) + k / 8] = (poison >> b) & 1 ? NAN : o;
            }
            // whole sectors: a thread writes a row of its own
            if (there && complete) {
#pragma unroll
                for (int k = 0; k < 32; k += 16) {
                    uint32_t h[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) h[q] = tc_bits<typename C::T>(v[k + 2 * q], v[k + 2 * q + 1]);
                    if (a.align >= 32) {
                        mx_put<8>(reinterpret_cast<uint8_t*>(out + 32 * b + k), h);
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            reinterpret_cast<uint16_t*>(out + 32 * b + k)[2 * q] = (uint16_t)h[q];
                            reinterpret_cast<uint16_t*>(out + 32 * b + k)[2 * q + 1] = (uint16_t)(h[q] >> 16);
                        }
                    }
                }
            } else if (there) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t h[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) h[q] = __float_as_uint(v[k + q]);
                    mx_put<8>(reinterpret_cast<uint8_t*>(part_row + 32 * b + k), h);
                }
            }
            __syncwarp();
        }
        if (there && !complete)
            *reinterpret_cast<float2*>(plan.rows + (int64_t)part * (TC_ROWS * (C::DIM + 2)) + TC_ROWS * C::DIM + 2 * (i * TC_TILE + r)) =
                make_float2(none ? -INFINITY : ref, l);
        else if (there && a.lse)
            a.lse[at * a.heads + head] = none ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;
        __syncwarp();
    }
}

// A piece's queries: rows as fp16 of a power of two times them, the largest in [2^14, 2^15), the sign of the softmax's scale with
// them; and what their scores are multiplied by, into buffer `parity`.  Warp `warp` of `warps` takes its share; ready() is called before
// anything is stored.
template <typename C, typename F>
__device__ __forceinline__ void tc_rows(const AttnArgs& a, const TcWalk& w, int warp, int warps, uint32_t parity, uint32_t base, uint8_t* smem, F ready) {
    constexpr int LANES = C::B <= 2 ? 8 : 16, ROWS = 32 / LANES, AT_ONCE = 4;
    const int lane = threadIdx.x & 31, u = lane % LANES, rows = w.p_seq.n * a.shared;
    const bool used = u < 4 * C::B;
    const typename C::T* const q = static_cast<const typename C::T*>(a.q) + w.p_seq.q0 * a.q_stride + (int64_t)w.p_head * a.shared * C::DIM + 8 * u;
    const float scale = fabsf(a.scale_log2), sign = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
    Raw8<typename C::T> next[AT_ONCE];
    const auto load = [&](int r0) {
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int row = min(w.p_tile * TC_ROWS + r0 + k * ROWS + lane / LANES, rows - 1), token = divided(row, a);
            next[k].w[0] = make_uint4(0, 0, 0, 0);
            if (used) raw_load(q + token * a.q_stride + (row - token * a.shared) * C::DIM, a.align, next[k]);
        }
    };
    if (warp * ROWS * AT_ONCE < TC_ROWS) load(warp * ROWS * AT_ONCE);
    ready();
    for (int r0 = warp * ROWS * AT_ONCE; r0 < TC_ROWS; r0 += warps * ROWS * AT_ONCE) {
        Raw8<typename C::T> raw[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) raw[k] = next[k];
        if (r0 + warps * ROWS * AT_ONCE < TC_ROWS) load(r0 + warps * ROWS * AT_ONCE);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int r = r0 + k * ROWS + lane / LANES;
            Row8 x;
            float v[8], top = 0.0f;
            raw_get(raw[k], x);
            x.get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 100);
            const float up = sign * two_to(14 - e);
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] *= up;
            if (used)
                sts128(base + C::Q + (r / TC_TILE) * C::Q_BYTES + (u / 8) * TC_TILE * 128 + (r % TC_TILE) * 128 + (((u & 7) ^ (r & 7)) << 4),
                       half2_bits(v[0], v[4]), half2_bits(v[1], v[5]), half2_bits(v[2], v[6]), half2_bits(v[3], v[7]));
            if (u == 0) *reinterpret_cast<float*>(smem + C::SCALE + (parity * TC_ROWS + r) * 4) = scale * two_to(e - 14);
        }
    }
    fence_async();
    __syncwarp();
}

// The loaders: the next piece's queries, as soon as the last scores of this one are done.  The first piece's are the softmax
// warps', who have nothing else to do yet.
template <typename C>
__device__ __forceinline__ void tc_queries(const AttnArgs& a, TcWalk w, const TcWaits& wait, uint32_t base, uint8_t* smem) {
    const int warp = (threadIdx.x >> 5) - TC_ISSUER - 1;
    uint32_t pieces = 0;
    while (true) {
        tc_next(a, w);
        if (!w.valid) return;
        if (w.g1 <= w.g0) continue;
        if (pieces > 0) {
            bool ok = true;
            tc_rows<C>(a, w, warp, TC_LOADERS, pieces & 1, base, smem, [&] { ok = wait(C::Q_FREE, (pieces - 1) & 1); });
            if (!ok) return;
            if ((threadIdx.x & 31) == 0) wait.arrive(C::Q_FULL);
        }
        ++pieces;
    }
}

template <typename C>
__global__ void __launch_bounds__(TC_THREADS, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;     // of the swizzled tiles
    uint8_t* const smem = smem_raw + (base - smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5;
    const TcWaits wait{base, reinterpret_cast<volatile int*>(smem + C::STOP), a.limit_ns};
    if (tid < C::BARS)
        mbar_init(base + tid * 8, (tid >= C::K_FULL && tid < C::K_EMPTY) || (tid >= C::V_FULL && tid < C::V_EMPTY) ? TC_DECODERS
                                  : tid == C::Q_FIRST ? 8 : tid == C::Q_FULL ? TC_LOADERS : tid >= C::P_FULL && tid < C::O_DONE ? 4 : 1);
    if (tid == 0) *wait.stop = 0;
    fence_mbar_init();
    if (warp == TC_ISSUER) tmem_alloc(base + C::TMEM, 512);
    pdl_trigger();
    pdl_wait();
    tc_fence_before();
    const TcWalk walk = tc_share(a, plan, reinterpret_cast<int64_t*>(smem + C::WORDS));     // with barriers of the block
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::TMEM);
    if (tid < 2) plan.parts[2 * blockIdx.x + tid].of = -1;
    __syncthreads();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TC_SOFTMAX_REGS));
        if (walk.left > 0) tc_softmax<C>(a, plan, walk, wait, base, smem, tmem);
    } else if (warp < TC_ISSUER) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_DECODE_REGS));
        if (walk.left > 0) tc_decode<C>(a, walk, wait, base, smem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_OTHER_REGS));
        if (walk.left > 0) {
            if (warp == TC_ISSUER) tc_issue<C>(a, walk, wait, base, tmem);
            else tc_queries<C>(a, walk, wait, base, smem);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == TC_ISSUER) tmem_dealloc(tmem, 512);
}

// Joins the parts of the pieces that were cut: block (w, y) 8 rows of the one that starts in worker w, a warp a row, 4 parts in
// flight at a time.
constexpr int TC_JOIN_WARPS = 8;

template <typename C>
__global__ void __launch_bounds__(TC_JOIN_WARPS * 32) join_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan) {
    constexpr int VEC = C::DIM / 32, AT_ONCE = 4;
    pdl_wait();
    const int w = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * TC_JOIN_WARPS + (threadIdx.x >> 5);
    const Part* parts = plan.parts;
    const int of = mx_ld(&parts[2 * w + 1].of), to0 = mx_ld(&parts[2 * w + 1].to);
    if (of < 0 || to0 >= of) return;                       // no piece starts here, or none that goes on
    const int s = mx_ld(&parts[2 * w + 1].seq), tile = mx_ld(&parts[2 * w + 1].tile), head = mx_ld(&parts[2 * w + 1].head);
    // the workers behind: whose first part ends the piece
    int n = 1;
    for (bool more = true; more; n += 32) {
        const int v = w + n + lane;
        const bool goes_on = v < plan.workers && mx_ld(&parts[2 * v].of) >= 0 && mx_ld(&parts[2 * v].to) < of;
        const uint32_t ends = __ballot_sync(0xffffffffu, !goes_on);
        more = !ends;
        if (ends) n += __ffs(ends) - 32;
    }
    n = min(n, plan.workers - w);
    const Seq seq = seq_of<TC_ROWS>(a, s, false);
    const int row = tile * TC_ROWS + r;
    if (row >= seq.n * a.shared) return;
    const auto rows_of = [&](int p) { return plan.rows + (p == 0 ? 2 * w + 1 : 2 * (w + p)) * (int64_t)(TC_ROWS * (C::DIM + 2)); };
    float ref = -INFINITY;
    for (int p = lane; p < n; p += 32) ref = larger(ref, mx_ld(rows_of(p) + TC_ROWS * C::DIM + 2 * r));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ref = larger(ref, __shfl_xor_sync(0xffffffffu, ref, d));
    float sum = 0.0f, v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
    for (int p0 = 0; p0 < n; p0 += AT_ONCE) {
        float k[AT_ONCE], l[AT_ONCE], x[AT_ONCE][VEC];
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const float* rows = rows_of(min(p0 + q, n - 1));
            k[q] = mx_ld(rows + TC_ROWS * C::DIM + 2 * r);
            l[q] = mx_ld(rows + TC_ROWS * C::DIM + 2 * r + 1);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] = mx_ld(rows + r * C::DIM + i * 32 + lane);
        }
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            if (p0 + q >= n) break;
            const float share = share_of(k[q], ref);
            sum = fmaf(share, l[q], sum);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = fmaf(share, x[q][i], v[i]);
        }
    }
    const float inv = ref == -INFINITY ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t)(seq.q0 + row / a.shared) * a.heads + head * a.shared + row % a.shared;
    uint16_t* out = static_cast<uint16_t*>(a.dst) + at * C::DIM;
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i * 32 + lane] = (uint16_t)tc_bits<typename C::T>(v[i] * inv, 0.0f);
    if (lane == 0 && a.lse) a.lse[at] = ref == -INFINITY ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <typename C>
q4q_status tc_run(const AttnArgs& a, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return cudaGetLastError(), Q4Q_ERR_CUDA;
    Plan plan;
    plan.workers = info.sm_count;
    plan.whole = 0;
    plan.least = 4;
    plan.parts = static_cast<Part*>(workspace);
    plan.rows = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + mx_up((int64_t)sizeof(Part) * 2 * plan.workers, 256));
    const q4q_status st = launch(attn_tc_kernel<C>, dim3((unsigned)plan.workers), TC_THREADS, C::BYTES, stream, a, plan);
    if (st != Q4Q_OK) return st;
    return launch(join_tc_kernel<C>, dim3((unsigned)plan.workers, TC_ROWS / TC_JOIN_WARPS), TC_JOIN_WARPS * 32, 0, stream, a, plan);
}

template <typename T>
q4q_status tc_run_type(const AttnArgs& a, int64_t head_dim, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    switch (head_dim) {
        case 64: return tc_run<Tc<2, T>>(a, workspace, stream, info);
        case 96: return tc_run<Tc<3, T>>(a, workspace, stream, info);
        default: return tc_run<Tc<4, T>>(a, workspace, stream, info);
    }
}

}  // namespace

size_t attn_tc_workspace(int64_t head_dim, const DeviceInfo& info) {
    return (size_t)(mx_up((int64_t)sizeof(Part) * 2 * info.sm_count, 256) + (int64_t)sizeof(float) * TC_ROWS * (head_dim + 2) * 2 * info.sm_count);
}

q4q_status attn_tc_run(const AttnArgs& a, int64_t head_dim, void* workspace, cudaStream_t stream, const DeviceInfo& info) {
    return a.type == Q4Q_TYPE_F16 ? tc_run_type<__half>(a, head_dim, workspace, stream, info)
                                  : tc_run_type<__nv_bfloat16>(a, head_dim, workspace, stream, info);
}

unsigned int attn_tc_take_device_status() { return attn_take_status_word(); }

}  // namespace q4q
