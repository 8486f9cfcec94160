// q4q_kv.cu -- keys and values into the paged 4-bit cache and out of it.
//
// Append: of token t's rows (keys normed and turned as q4q_rope.cu has them, values as they are) each
// block of 32 becomes Q4_0: d = amax / 8, code = round(x / d) half away from zero, limited to
// [-8, 7], plus 8 -- the encoder of q4q_common.cuh, fed from registers, so a key's fp32 values never
// go to memory.  Rows are limited to +-65504 first: the scale is then at most 8188 and every
// (code - 8) d is finite in fp16, which the attention's tensor-core form decodes to.  A block with an
// infinity or a NaN gets the scale NaN and codes of 8.
//
// Rows, lanes and warps as in q4q_rope.cu: a lane's 8 values are one word of key codes or two halves of value codes.  The
// order of the cache (q4q_attn.cuh) spreads a value row's bytes over its octet's 4 D bytes; a prompt's neighbours fill the
// gaps while the lines are in L2.  Measured in a graph, keys and values of 8 heads of 128: one fp32 token 3.1 us (launch and
// two loads in a row), 8192 bf16 tokens with norm and rotation 29.3 us, without 19.8 us; 43 MB are moved, so 1.5 and
// 2.2 TB/s.  Half of the warps keep to keys, half to values, so with norm and rotation the values' are done well before the
// keys'; the encoder's 45 instructions for 8 codes are a fraction of either time at full issue.  The row
// gather of 8192 slots: 13.7 us (3.1 TB/s), on append's grid: 16 of the 32 warps an SM that its 56 registers would let in.
#include <algorithm>

#include "q4q_attn.cuh"
#include "q4q_mx_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_kv_status = 0;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int SLOTS = 4;           // row slots (of 32 / LANES rows) that a warp takes at a time

struct KvArgs {
    const void *k, *v;
    uint8_t* cache;
    const float* w;
    const float* table;
    const int32_t *pos, *slots;
    void *k_dst, *v_dst;
    int64_t k_stride, v_stride, n_pos, n_tokens, n_slots;     // n_slots: of the cache
    int heads, dim, rot, halves, align, page_log;
    float eps;
    float2 inv_dim;
    int per, items;                // times SLOTS row slots that a warp takes of one side (keys or values) of a token; warps a side
    int tokens_at_once;            // of the grid's warps, 2 * items of them a token
};

constexpr float KV_MAX = 65504.0f;

// The word of a lane's 8 codes (element e at bit 4 e), all 32 lanes together: what pack_q4_word of q4q_common.cuh gives, in
// two-lane instructions, about 45 of them.  t = x rcp(d) is stopped at 7 and rounded by adding 1.5 2^23 + 8, which leaves
// code + 8 in the low bits; the constant above them leaves with one subtraction from the sum of all 8, each at its place.
//
// `raw`: the values are of a 16-bit type (or +-65504).  Their quotients hit half-integers often, and 8 bf16 rows out of 10 would
// take the divisions below.  But x and amax have 11-bit mantissas, so a quotient that is no half-integer h is at least h / 2^15 away
// from one: with the reciprocal made 2^-20 larger (its error and the product's are 2^-22), ties, and they alone, come out
// just beyond it, where rounding to nearest takes them away from zero, as the code is defined.  (8192 tokens of 8 heads of
// 128, bf16 keys and values: 31 us with the divisions, 20 without.)
// Otherwise, as there: t rounds as the IEEE quotient does, but within 5e-5 of a half-integer, where that is computed.
__device__ __forceinline__ uint32_t code_word(const float (&v)[8], float d, bool raw) {
    // d = 0 (zeros, lanes past a row's end): quotients of 0, whose code is 8 as defined, so that its warp's other blocks stay on this way.
    // (Heads of 96, which leave 4 lanes of 16 empty, 8192 bf16 tokens: 35.6 us where d = 0 took the other way, 19.5 so; 5 heads of 128 23.8, 18.0.)
    float inv = d == 0.0f ? 0.0f : recip_approx(d);
    const bool sure = raw && __all_sync(0xffffffffu, inv < 1e38f);           // a subnormal d takes the other way
    if (sure) inv = fmaf(inv, 9.5367431640625e-7f, inv);
    constexpr float MAGIC = 12582920.0f;                   // 0x4B400008
    uint32_t w = 0;
    float far = 0.0f;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        float t0, t1, r0, r1, e0, e1;
        unpack2(fmul2(pack2(v[2 * i], v[2 * i + 1]), pack2(inv, inv)), t0, t1);
        // NaN stays (fmin would drop it)
        t0 = t0 > 7.0f ? 7.0f : t0;
        t1 = t1 > 7.0f ? 7.0f : t1;
        const uint64_t t = pack2(t0, t1), rm = fadd2(t, pack2(MAGIC, MAGIC));
        unpack2(rm, r0, r1);
        unpack2(fsub2(t, fsub2(rm, pack2(MAGIC, MAGIC))), e0, e1);
        far = max3_abs(far, e0, e1);
        w = (w * 16 + __float_as_uint(r1)) * 16 + __float_as_uint(r0);
    }
    w -= 0x4B400000u * 0x11111111u;
    const bool near = !sure && !(far <= NEAR_LIMIT);
    if (__any_sync(0xffffffffu, near)) {
        if (near) {
            w = 0;
#pragma unroll
            for (int e = 7; e >= 0; --e) w = w * 16 + (uint32_t)(quant_one(v[e], d, -8.0f, 7.0f) + 8);
        }
    }
    return w;
}

// A lane's 8 values of a block of 32 (4 lanes): the word of codes, and in d_bits the block's scale.
__device__ __forceinline__ uint32_t encode_block(const Row8& x, bool raw, uint16_t& d_bits) {
    float v[8], m = 0.0f;
    x.get(v);
#pragma unroll
    for (int e = 0; e < 8; e += 2) m = max3_abs(m, v[e], v[e + 1]);                        // NaN if one is
    m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.0f);
    m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, 2), 0.0f);
    const bool finite = m <= 3.402823466e38f;
    if (__any_sync(0xffffffffu, !(m <= KV_MAX))) {
        if (!(m <= KV_MAX)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = finite ? fminf(fmaxf(v[e], -KV_MAX), KV_MAX) : 0.0f;
            m = finite ? KV_MAX : 0.0f;
        }
    }
    const float d = scale_q4(m);
    const uint32_t word = code_word(v, d, raw);
    d_bits = finite ? fp16_bits(d) : 0x7fffu;
    return word;
}

// A warp's side and heads, the same through all of its tokens (as in q4q_rope.cu).
struct Place {
    bool value;
    int row0;
    int64_t token;
};

template <int LANES>
__device__ __forceinline__ Place place_of(const KvArgs& a) {
    const int id = blockIdx.x * WARPS + (threadIdx.x >> 5), item = id % (2 * a.items);
    Place p;
    p.value = item >= a.items;
    p.row0 = (p.value ? item - a.items : item) * a.per * SLOTS * (32 / LANES) + (threadIdx.x & 31) / LANES;
    p.token = id / (2 * a.items);
    if (p.token >= a.tokens_at_once) p.token = a.n_tokens;           // warps that are left over
    return p;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(THREADS, 2) append_kernel(const __grid_constant__ KvArgs a) {
    constexpr int ROWS = 32 / LANES;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, in_row = lane % LANES, at = in_row * 8, b = in_row >> 2, t = in_row & 3;
    const bool used = at < a.dim;
    Place p = place_of<LANES>(a);
    const bool turns = a.table && !p.value, norm = a.w && !p.value;
    Row8 w;
    w.clear();
    if (norm && used) {
        Raw8<float> r;
        raw_load(a.w + at, 16, r);
        raw_get(r, w);
    }
    Turn turning;
    turn_init(turning, a.rot, a.halves, used ? at : a.rot);
    constexpr bool AHEAD = sizeof(T) == 2;                           // the next step's rows are loaded before this one's are used
    Raw8<T> in[SLOTS];
    const auto load = [&](int64_t of, int row) {
        const T* x_row = (p.value ? static_cast<const T*>(a.v) + of * a.v_stride : static_cast<const T*>(a.k) + of * a.k_stride) + at;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            in[i] = Raw8<T>{};
            if (row + i * ROWS < a.heads && used) raw_load(x_row + (int64_t)(row + i * ROWS) * a.dim, a.align, in[i]);
        }
    };
    int next_slot = -1, next_pos = 0;
    if (p.token < a.n_tokens) {
        next_slot = mx_ld(a.slots + p.token);
        if (a.table) next_pos = mx_ld(a.pos + p.token);
        if (AHEAD) load(p.token, p.row0);
    }
    for (; p.token < a.n_tokens; p.token += a.tokens_at_once) {
        const int slot = next_slot, pos = next_pos;
        const int64_t page = slot >> a.page_log, next = p.token + a.tokens_at_once;
        const int group = (slot >> 4) & ((1 << (a.page_log - 4)) - 1), i16 = slot & 15;
        const bool bad = slot >= a.n_slots || (a.table && (pos < 0 || pos >= a.n_pos));
        const bool known = slot >= 0 && !bad;
        if (slot >= 0 && bad && lane == 0) record_error(&g_kv_status, Q4Q_ERR_ARG);
        if (known && turns) turn_load(turning, a.table + (int64_t)pos * a.rot, a.rot, a.halves, at, false);
        if (next < a.n_tokens) {
            next_slot = mx_ld(a.slots + next);
            if (a.table) next_pos = mx_ld(a.pos + next);
        }
        for (int k = 0; k < a.per; ++k) {
            const int row = p.row0 + k * SLOTS * ROWS;
            if (row - lane / LANES >= a.heads) break;
            if (!AHEAD && known) load(p.token, row);
            Row8 v[SLOTS];
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) raw_get(in[i], v[i]);
            if (AHEAD) {
                const bool more = k + 1 < a.per && row - lane / LANES + SLOTS * ROWS < a.heads;
                if (more) load(p.token, row + SLOTS * ROWS);
                else if (next < a.n_tokens) load(next, p.row0);
            }
            if (!known) continue;
            if (norm) {
                float r[SLOTS];
                inverse_norm4<LANES, sizeof(T) == 2>(v, a.inv_dim, a.eps, r);
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i].p[j] = fmul2(fmul2(v[i].p[j], pack2(r[i], r[i])), w.p[j]);
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (turns) turn(v[i], turning, a.halves);
                uint16_t d;
                const uint32_t word = encode_block(v[i], sizeof(T) == 2 && !norm && !turns, d);
                const int head = row + i * ROWS;
                if (head < a.heads && used) {
                    uint8_t* chunk = a.cache + kv_chunk_offset(page, head, group, a.heads, a.page_log, a.dim);
                    if (p.value) {
                        *reinterpret_cast<uint16_t*>(chunk + kv_v_half(i16, 2 * t, b, a.dim)) = (uint16_t)word;
                        *reinterpret_cast<uint16_t*>(chunk + kv_v_half(i16, 2 * t + 1, b, a.dim)) = (uint16_t)(word >> 16);
                    } else {
                        *reinterpret_cast<uint32_t*>(chunk + kv_k_word(i16, t, b, a.dim)) = word;
                    }
                    if (t == 0) *reinterpret_cast<uint16_t*>(chunk + kv_scale(p.value, i16, b, a.dim)) = d;
                }
            }
        }
    }
}

template <typename T, int LANES>
__global__ void __launch_bounds__(THREADS, 2) get_rows_kernel(const __grid_constant__ KvArgs a) {
    constexpr int ROWS = 32 / LANES;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, in_row = lane % LANES, at = in_row * 8, b = in_row >> 2, t = in_row & 3;
    const bool used = at < a.dim;
    Place p = place_of<LANES>(a);
    void* const dst = p.value ? a.v_dst : a.k_dst;
    int slot = p.token < a.n_tokens ? mx_ld(a.slots + p.token) : -1;
    for (; p.token < a.n_tokens; p.token += a.tokens_at_once) {
        const bool known = slot >= 0 && slot < a.n_slots;
        if (slot >= a.n_slots && lane == 0) record_error(&g_kv_status, Q4Q_ERR_ARG);
        const int64_t page = known ? slot >> a.page_log : 0;
        const int group = (slot >> 4) & ((1 << (a.page_log - 4)) - 1), i16 = slot & 15;
        const int64_t next = p.token + a.tokens_at_once;
        if (next < a.n_tokens) slot = mx_ld(a.slots + next);
        if (!dst) continue;
        T* to = static_cast<T*>(dst) + p.token * a.heads * (int64_t)a.dim + at;
        for (int k = 0; k < a.per; ++k) {
            const int row = p.row0 + k * SLOTS * ROWS;
            if (row - lane / LANES >= a.heads) break;
            uint32_t word[SLOTS];
            uint16_t d[SLOTS];
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                const int head = row + i * ROWS;
                word[i] = 0x88888888u;
                d[i] = 0;
                if (head < a.heads && used && known) {
                    const uint8_t* chunk = a.cache + kv_chunk_offset(page, head, group, a.heads, a.page_log, a.dim);
                    if (p.value)
                        word[i] = (uint32_t)mx_ld(reinterpret_cast<const uint16_t*>(chunk + kv_v_half(i16, 2 * t, b, a.dim))) |
                                  (uint32_t)mx_ld(reinterpret_cast<const uint16_t*>(chunk + kv_v_half(i16, 2 * t + 1, b, a.dim))) << 16;
                    else
                        word[i] = mx_ld(reinterpret_cast<const uint32_t*>(chunk + kv_k_word(i16, t, b, a.dim)));
                    d[i] = mx_ld(reinterpret_cast<const uint16_t*>(chunk + kv_scale(p.value, i16, b, a.dim)));
                }
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (row + i * ROWS >= a.heads || !used) continue;
                // (code - 8) in fp16 is exact, elements e and e + 4 side by side
                const uint4 h = nibbles_to_f16x8(word[i]);
                const uint32_t hh[4] = {h.x, h.y, h.z, h.w};
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh[e]));
                    v[e] = f.x, v[e + 4] = f.y;
                }
                const float scale = fp16_to_f32(d[i]);
                Row8 x;
                x.set(v);
#pragma unroll
                for (int e = 0; e < 4; ++e) x.p[e] = fmul2(x.p[e], pack2(scale, scale));
                row_store(to + (int64_t)(row + i * ROWS) * a.dim, a.align, x);
            }
        }
    }
}

// As q4q_rope.cu's: as many heads of a token to a warp as leave every SM the warps that it holds.
int plan(KvArgs& a, int lanes, const DeviceInfo& info) {
    const int64_t warps = (int64_t)info.sm_count * 2 * WARPS;
    const int rows = SLOTS * 32 / lanes;
    a.per = 1;
    a.items = (a.heads + rows - 1) / rows;
    while (a.items > 1) {
        const int fewer = (a.heads + rows * 2 * a.per - 1) / (rows * 2 * a.per);
        if (a.n_tokens * 2 * fewer < warps) break;
        a.per *= 2;
        a.items = fewer;
    }
    a.tokens_at_once = (int)std::max<int64_t>(1, std::min<int64_t>(a.n_tokens, warps / (2 * a.items)));
    return (a.tokens_at_once * 2 * a.items + WARPS - 1) / WARPS;
}

template <typename K>
q4q_status launch(K kernel, const KvArgs& a, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? launch_status() : (cudaGetLastError(), Q4Q_ERR_CUDA);
}

template <typename T, int LANES>
q4q_status run_t(KvArgs& a, bool append, cudaStream_t stream, const DeviceInfo& info) {
    const int blocks = plan(a, LANES, info);
    return append ? launch(append_kernel<T, LANES>, a, blocks, stream) : launch(get_rows_kernel<T, LANES>, a, blocks, stream);
}

template <typename T>
q4q_status run_lanes(KvArgs& a, bool append, cudaStream_t stream, const DeviceInfo& info) {
    return a.dim <= 64 ? run_t<T, 8>(a, append, stream, info) : a.dim <= 128 ? run_t<T, 16>(a, append, stream, info) : run_t<T, 32>(a, append, stream, info);
}

q4q_status run(KvArgs& a, int type, bool append, cudaStream_t stream) {
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    switch (type) {
        case Q4Q_TYPE_F32: return run_lanes<float>(a, append, stream, info);
        case Q4Q_TYPE_F16: return run_lanes<__half>(a, append, stream, info);
        default: return run_lanes<__nv_bfloat16>(a, append, stream, info);
    }
}

}  // namespace

unsigned int kv_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_kv_status, &z, sizeof(z));
    return v;
}

q4q_status kv_check(int64_t n_pages, int page_tokens, int n_kv_heads, int64_t head_dim, int& page_log) {
    if (!kv_dim_ok(head_dim) || !kv_page_ok(page_tokens) || n_kv_heads < 1 || n_kv_heads > 1024 || n_pages < 0) return Q4Q_ERR_SHAPE;
    if ((int64_t)n_kv_heads * head_dim * page_tokens / 8 * 9 >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (n_pages >= (1ll << 31) / page_tokens) return Q4Q_ERR_SHAPE;
    page_log = 4;
    while ((1 << page_log) < page_tokens) ++page_log;
    return Q4Q_OK;
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_kv_page_size(int n_kv_heads, int64_t head_dim, int page_tokens, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    int page_log;
    const q4q_status st = kv_check(0, page_tokens, n_kv_heads, head_dim, page_log);
    if (st != Q4Q_OK) return st;
    *bytes = (size_t)n_kv_heads * (page_tokens / KV_GROUP) * kv_chunk_bytes((int)head_dim);
    return Q4Q_OK;
}

extern "C" q4q_status q4q_kv_append(void* cache, int64_t n_pages, int page_tokens, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, int type, int n_kv_heads, int64_t head_dim, int64_t n_tokens, const int32_t* slots,
                                    const float* k_weight, float eps, const float* table, int64_t n_pos, int rot, int mode,
                                    const int32_t* pos, q4q_stream_t stream) {
    KvArgs a{};
    const q4q_status st = kv_check(n_pages, page_tokens, n_kv_heads, head_dim, a.page_log);
    if (st != Q4Q_OK) return st;
    const int64_t width = n_kv_heads * head_dim;
    if (n_tokens < 0 || n_tokens >= (1ll << 31) || n_pos < 0 || n_pos >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (k_stride < width || v_stride < width || k_stride >= (1ll << 31) || v_stride >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (table && (rot <= 0 || rot % 16 || rot > head_dim)) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(type) || (mode != Q4Q_ROPE_PAIRS && mode != Q4Q_ROPE_HALVES) || !(eps >= 0.0f)) return Q4Q_ERR_ARG;
    if (n_tokens == 0) return Q4Q_OK;
    if (!cache || !k || !v || !slots || (table && !pos)) return Q4Q_ERR_NULL;
    const size_t size = mx_type_bytes(type);
    if (!aligned(cache, 16) || !aligned(k, size) || !aligned(v, size) || !aligned(slots, 4) || (k_weight && !aligned(k_weight, 16)) ||
        (table && (!aligned(table, 16) || !aligned(pos, 4))))
        return Q4Q_ERR_ALIGN;
    a.k = k;
    a.v = v;
    a.cache = static_cast<uint8_t*>(cache);
    a.w = k_weight;
    a.table = table;
    a.pos = pos;
    a.slots = slots;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n_pos = n_pos;
    a.n_tokens = n_tokens;
    a.n_slots = n_pages * page_tokens;
    a.heads = n_kv_heads;
    a.dim = (int)head_dim;
    a.rot = table ? rot : 0;
    a.halves = mode == Q4Q_ROPE_HALVES;
    a.align = aligned(k, 16) && aligned(v, 16) && k_stride * size % 16 == 0 && v_stride * size % 16 == 0 ? 16 : 1;
    a.eps = eps;
    const double inv = 1.0 / (double)head_dim;
    a.inv_dim = make_float2((float)inv, (float)(inv - (double)(float)inv));
    return run(a, type, true, (cudaStream_t)stream);
}

extern "C" q4q_status q4q_kv_get_rows(const void* cache, int64_t n_pages, int page_tokens, int n_kv_heads, int64_t head_dim,
                                      const int32_t* slots, int64_t n_slots, void* k_dst, void* v_dst, int dst_type, q4q_stream_t stream) {
    KvArgs a{};
    const q4q_status st = kv_check(n_pages, page_tokens, n_kv_heads, head_dim, a.page_log);
    if (st != Q4Q_OK) return st;
    if (n_slots < 0 || n_slots >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(dst_type)) return Q4Q_ERR_ARG;
    if (n_slots == 0 || (!k_dst && !v_dst)) return Q4Q_OK;
    if (!cache || !slots) return Q4Q_ERR_NULL;
    const size_t size = mx_type_bytes(dst_type);
    if (!aligned(cache, 16) || !aligned(slots, 4) || !aligned(k_dst, size) || !aligned(v_dst, size)) return Q4Q_ERR_ALIGN;
    a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
    a.slots = slots;
    a.k_dst = k_dst;
    a.v_dst = v_dst;
    a.n_tokens = n_slots;
    a.n_slots = n_pages * page_tokens;
    a.heads = n_kv_heads;
    a.dim = (int)head_dim;
    a.align = aligned(k_dst, 16) && aligned(v_dst, 16) ? 16 : 1;
    return run(a, dst_type, false, (cudaStream_t)stream);
}
