// q4q_rope.cu -- norms of queries and keys for each head with the position rotation in the same
// pass, its backward pass, and the table of cosines and sines.
//
// Of one head's row x (D values) of a token at position p, with w optional:
//   r = 1 / sqrt(mean(x^2) + eps),  z = (x r) w,  y = R_p z
// R_p turns the pairs (a, b) of z's first rot values, (z_i, z_{i + rot/2}) or (z_2i, z_2i+1), by the
// angle of the table's row p: a' = a c - b s, b' = b c + a s.  Backward, dz = R_p^T dy:
//   dx = r (dz w - xh mean(dz w xh)), xh = x r;   dw = sum over tokens and heads of dz xh
// Everything is fp32; r is that of 64-bit sums (inverse_norm), the rest rounds each product and sum.
//
// A row takes D / 8 lanes, 8 values each.  A warp keeps to one side (queries or keys) and one run of heads through all of
// its tokens, so weights and places are looked up once, and takes 4 row slots at a time (2 backward), whose loads
// are in flight together and whose norms share their sums' last steps and root.  Few tokens are bound by the
// launch and two loads behind one another.  dw is summed in registers over a warp's rows, then
// over the block's warps, and the blocks' sums by a second kernel in the order of the blocks: no atomics, results do
// not vary.
//
// Measured in a graph (32 + 8 heads of 128): one token 3.5 us; 8191 bf16 tokens forward 49.2 us (168 MB, 3.4 TB/s), backward with both
// weights 77 us (252 MB, 3.3 TB/s).  What that is made of: neither norm nor rotation, a copy, 29 us (5.8 TB/s), the norm alone 32, the rotation
// alone 43: a token's angles are loaded when it is its turn, and each value's partner is fetched from another lane.  Backward 38, 51, 54.
// fp32: 67, 73, 75, both 83.  (Three blocks an SM with fewer registers were slower, 57.7.)
#include <algorithm>

#include "q4q_attn.cuh"
#include "q4q_mx_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_rope_status = 0;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int FORWARD_SLOTS = 4, BACK_SLOTS = 2;   // row slots (of 32 / LANES rows) that a warp takes at a time

struct Side {                      // the queries, or the keys
    const void* x;                 // [tokens][heads][D], rows of a token at `stride` elements
    const void* dy;
    const float* w;
    void* out;                     // [tokens][heads][D]: y, or dx
    int64_t stride;
    int heads;
    int items;                     // warps that share a token's heads
    int per;                       // times SLOTS row slots that each of them takes
};

struct RopeArgs {
    Side side[2];
    const float* table;
    const int32_t* pos;
    int64_t n_pos, n_tokens;
    int dim, rot, halves, align;
    float eps;
    float2 inv_dim;
    int tokens_at_once;            // of the grid's warps, side[0].items + side[1].items of them a token
    float* partial;                // backward: [blocks][2][D]
};

template <typename T, int LANES, bool BACK>
__global__ void __launch_bounds__(THREADS, 2) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int ROWS = 32 / LANES, SLOTS = BACK ? BACK_SLOTS : FORWARD_SLOTS;
    extern __shared__ float sums[];            // backward: [warps][2][D]
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % LANES * 8;
    const bool used = at < a.dim;
    const int items = a.side[0].items + a.side[1].items, id = blockIdx.x * WARPS + warp;
    const int item = id % items, which = item >= a.side[0].items;
    const Side& s = a.side[which];
    const int row0 = (which ? item - a.side[0].items : item) * s.per * SLOTS * ROWS + lane / LANES;
    const bool norm = s.w != nullptr;
    Row8 w, dw;
    w.clear();
    dw.clear();
    if (norm && used) {
        Raw8<float> r;
        raw_load(s.w + at, 16, r);
        raw_get(r, w);
    }
    Turn turning;
    turn_init(turning, a.rot, a.halves, used ? at : a.rot);
    int64_t token = id / items;
    if (token >= a.tokens_at_once) token = a.n_tokens;               // warps that are left over
    constexpr bool AHEAD = sizeof(T) == 2;                           // the next step's rows are loaded before this one's are used
    const bool reads_x = !BACK || norm;
    Raw8<T> in[SLOTS], grad[BACK ? SLOTS : 1];
    const auto load = [&](int64_t of, int row) {
        const T* x_row = static_cast<const T*>(s.x) + of * s.stride + at;
        const T* g_row = static_cast<const T*>(s.dy) + of * s.heads * (int64_t)a.dim + at;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int head = row + i * ROWS;
            in[i] = Raw8<T>{};
            if constexpr (BACK) grad[i] = Raw8<T>{};
            if (head < s.heads && used) {
                if (reads_x) raw_load(x_row + (int64_t)head * a.dim, a.align, in[i]);
                if constexpr (BACK) raw_load(g_row + (int64_t)head * a.dim, a.align, grad[i]);
            }
        }
    };
    int pos = 0, pos_next = 0;
    if (token < a.n_tokens) {
        if (a.table) pos_next = mx_ld(a.pos + token);
        if (AHEAD) load(token, row0);
    }
    for (; token < a.n_tokens; token += a.tokens_at_once) {
        T* out_row = static_cast<T*>(s.out) + token * s.heads * (int64_t)a.dim + at;
        const int64_t next = token + a.tokens_at_once;
        pos = pos_next;
        const bool known = !a.table || (pos >= 0 && pos < a.n_pos);
        if (a.table) {
            if (known) turn_load(turning, a.table + (int64_t)pos * a.rot, a.rot, a.halves, at, BACK);
            else if (lane == 0) record_error(&g_rope_status, Q4Q_ERR_ARG);
            if (next < a.n_tokens) pos_next = mx_ld(a.pos + next);
        }
        for (int k = 0; k < s.per; ++k) {
            const int row = row0 + k * SLOTS * ROWS;
            if (row - lane / LANES >= s.heads) break;
            if (!AHEAD) load(token, row);
            Row8 v[SLOTS], g[BACK ? SLOTS : 1];
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                raw_get(in[i], v[i]);
                if constexpr (BACK) raw_get(grad[i], g[i]);
            }
            if (AHEAD) {
                const bool more = k + 1 < s.per && row - lane / LANES + SLOTS * ROWS < s.heads;
                if (more) load(token, row + SLOTS * ROWS);
                else if (next < a.n_tokens) load(next, row0);
            }
            if constexpr (!BACK) {
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
                    if (a.table) turn(v[i], turning, a.halves);
                    const int head = row + i * ROWS;
                    if (!known) v[i].clear();
                    if (head < s.heads && used) row_store(out_row + (int64_t)head * a.dim, a.align, v[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < SLOTS; ++i) {
                    if (a.table) turn(g[i], turning, a.halves);
                    if (!known) g[i].clear();
                    if (norm) {
                        // sums of x^2, and of dz w x, over the row
                        uint64_t sq = 0, dot = 0;
                        Row8 dh;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            dh.p[j] = fmul2(g[i].p[j], w.p[j]);
                            sq = ffma2(v[i].p[j], v[i].p[j], sq);
                            dot = ffma2(dh.p[j], v[i].p[j], dot);
                        }
                        float s0, s1, d0, d1;
                        unpack2(sq, s0, s1);
                        unpack2(dot, d0, d1);
                        s0 += s1, d0 += d1;
#pragma unroll
                        for (int d = 1; d < LANES; d <<= 1) {
                            s0 += __shfl_xor_sync(0xffffffffu, s0, d);
                            d0 += __shfl_xor_sync(0xffffffffu, d0, d);
                        }
                        // 0 where this lane holds no row: eps may be 0
                        const float r = known && row + i * ROWS < s.heads ? rsqrtf(s0 * a.inv_dim.x + a.eps) : 0.0f;
                        const float back = -(d0 * a.inv_dim.x) * r * r;               // of x: dx = r (dh - x mean(dh x) r^2)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            dw.p[j] = ffma2(g[i].p[j], fmul2(v[i].p[j], pack2(r, r)), dw.p[j]);
                            g[i].p[j] = fmul2(ffma2(v[i].p[j], pack2(back, back), dh.p[j]), pack2(r, r));
                        }
                    }
                    const int head = row + i * ROWS;
                    if (head < s.heads && used) row_store(out_row + (int64_t)head * a.dim, a.align, g[i]);
                }
            }
        }
    }
    if constexpr (BACK) {
        if (!a.partial) return;
        // the warp's rows, then the block's warps
        float mine[8];
        dw.get(mine);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int d = LANES; d < 32; d <<= 1) mine[e] += __shfl_xor_sync(0xffffffffu, mine[e], d);
            if (lane < LANES && used) {
                sums[(warp * 2 + which) * a.dim + at + e] = mine[e];
                sums[(warp * 2 + !which) * a.dim + at + e] = 0.0f;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.dim; i += THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) v += sums[k * 2 * a.dim + i];
            a.partial[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
        }
    }
}

// One block for 8 columns of the blocks' sums: 32 threads a column, each adds every 32nd.
__global__ void __launch_bounds__(THREADS) weight_sum_kernel(const float* partial, int blocks, int dim, float* dwq, float* dwk) {
    pdl_wait();
    const int col = blockIdx.x * WARPS + (threadIdx.x & (WARPS - 1)), part = threadIdx.x / WARPS;   // 32 parts, 8 columns side by side
    __shared__ float sums[32][WARPS + 1];
    float v = 0.0f;
    if (col < 2 * dim)
        for (int b = part; b < blocks; b += 32) v += mx_ld(partial + (int64_t)b * 2 * dim + col);
    sums[part][threadIdx.x & (WARPS - 1)] = v;
    __syncthreads();
    if (threadIdx.x < WARPS && col < 2 * dim) {
        float* to = col < dim ? dwq : dwk;
        if (to) {
            float s = 0.0f;
            for (int p = 0; p < 32; ++p) s += sums[p][threadIdx.x];
            to[col < dim ? col : col - dim] = s;
        }
    }
}

// cos and sin of p base^(-2i / rot), in 64 bits
__global__ void __launch_bounds__(THREADS) rope_table_kernel(float* table, int64_t n_pos, int rot, double base) {
    const int half = rot / 2;
    for (int64_t i = blockIdx.x * (int64_t)THREADS + threadIdx.x; i < n_pos * half; i += (int64_t)gridDim.x * THREADS) {
        const int64_t p = i / half;
        const int k = (int)(i - p * half);
        double s, c;
        sincos((double)p * pow(base, -2.0 * k / rot), &s, &c);
        table[p * rot + k] = (float)c;
        table[p * rot + half + k] = (float)s;
    }
}

constexpr int BLOCKS_PER_SM = 2;   // that 128 registers a thread leave

// The grid, and how many warps share a token's heads.  A warp that takes more heads of a token loads its angles fewer
// times, but few tokens should use all SMs: as many heads as leave every SM the warps of the blocks it holds.  All of the
// grid's warps then walk on by the same number of tokens.
int plan(RopeArgs& a, int lanes, int slots, const DeviceInfo& info) {
    const int64_t warps = (int64_t)info.sm_count * BLOCKS_PER_SM * WARPS;
    const int rows = slots * 32 / lanes;
    const int heads = a.side[0].heads + a.side[1].heads;
    int items = 0;
    for (int per = 1;; per *= 2) {
        int sum = 0;
        for (const Side& s : a.side) sum += (s.heads + rows * per - 1) / (rows * per);
        // no further where too few warps would be left with work, or where warps would have less to do than others
        if (per > 1 && (sum == items || a.n_tokens * sum < warps || (int64_t)sum * per * rows * 8 > heads * 9)) break;
        items = sum;
        for (Side& s : a.side) {
            s.per = per;
            s.items = (s.heads + rows * per - 1) / (rows * per);
        }
    }
    const int64_t at_once = std::max<int64_t>(1, std::min<int64_t>(a.n_tokens, warps / items));
    a.tokens_at_once = (int)at_once;
    return (int)((at_once * items + WARPS - 1) / WARPS);
}

template <typename... Params, typename... Args>
q4q_status launch(void (*kernel)(Params...), int grid, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
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

int lanes_of(int64_t dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// A backward call's workspace has one row of sums for each block; with up to 2048 heads a token may take more warps than
// the SMs hold.
int back_blocks(const DeviceInfo& info) { return std::max(info.sm_count * BLOCKS_PER_SM, 2 * 1024 / (BACK_SLOTS * WARPS)) + 1; }

template <typename T, int LANES>
q4q_status run_t(RopeArgs& a, bool back, cudaStream_t stream, const DeviceInfo& info, int& blocks) {
    blocks = plan(a, LANES, back ? BACK_SLOTS : FORWARD_SLOTS, info);
    if (!back) return launch(norm_rope_kernel<T, LANES, false>, blocks, 0, stream, a);
    return launch(norm_rope_kernel<T, LANES, true>, blocks, a.partial ? sizeof(float) * WARPS * 2 * a.dim : 0, stream, a);
}

template <typename T>
q4q_status run_lanes(RopeArgs& a, bool back, cudaStream_t stream, const DeviceInfo& info, int& blocks) {
    switch (lanes_of(a.dim)) {
        case 8: return run_t<T, 8>(a, back, stream, info, blocks);
        case 16: return run_t<T, 16>(a, back, stream, info, blocks);
        default: return run_t<T, 32>(a, back, stream, info, blocks);
    }
}

q4q_status run(RopeArgs& a, int type, bool back, cudaStream_t stream, const DeviceInfo& info, int& blocks) {
    switch (type) {
        case Q4Q_TYPE_F32: return run_lanes<float>(a, back, stream, info, blocks);
        case Q4Q_TYPE_F16: return run_lanes<__half>(a, back, stream, info, blocks);
        default: return run_lanes<__nv_bfloat16>(a, back, stream, info, blocks);
    }
}

// What forward and backward check alike; empty: nothing to do.
q4q_status check(RopeArgs& a, int type, int64_t head_dim, int64_t n_tokens, const float* table, int64_t n_pos, int rot, int mode,
                 const int32_t* pos, float eps, bool back, bool& empty) {
    empty = false;
    if (!kv_dim_ok(head_dim) || n_tokens < 0 || n_tokens >= (1ll << 31) || n_pos < 0 || n_pos >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    for (const Side& s : a.side) {
        if (s.heads < 0 || s.heads > 1024) return Q4Q_ERR_SHAPE;
        if (s.heads > 0 && (s.stride < s.heads * head_dim || s.stride >= (1ll << 31))) return Q4Q_ERR_SHAPE;
    }
    if (!mx_type_ok(type) || (mode != Q4Q_ROPE_PAIRS && mode != Q4Q_ROPE_HALVES) || !(eps >= 0.0f)) return Q4Q_ERR_ARG;
    if (table && (rot <= 0 || rot % 16 || rot > head_dim)) return Q4Q_ERR_SHAPE;
    empty = n_tokens == 0 || a.side[0].heads + a.side[1].heads == 0;
    if (empty) return Q4Q_OK;
    if (table && !pos) return Q4Q_ERR_NULL;
    if ((table && !aligned(table, 16)) || (pos && !aligned(pos, 4))) return Q4Q_ERR_ALIGN;
    const size_t size = mx_type_bytes(type);
    a.align = 16;
    for (const Side& s : a.side) {
        if (!s.heads) continue;
        const bool reads_x = !back || s.w;
        if ((reads_x && !s.x) || !s.out || (back && !s.dy)) return Q4Q_ERR_NULL;
        if (!aligned(s.x, size) || !aligned(s.out, size) || (s.dy && !aligned(s.dy, size)) || (s.w && !aligned(s.w, 16))) return Q4Q_ERR_ALIGN;
        if (!aligned(s.x, 16) || !aligned(s.out, 16) || (back && !aligned(s.dy, 16)) || s.stride * size % 16) a.align = 1;
    }
    a.table = table;
    a.pos = pos;
    a.n_pos = n_pos;
    a.n_tokens = n_tokens;
    a.dim = (int)head_dim;
    a.rot = table ? rot : 0;
    a.halves = mode == Q4Q_ROPE_HALVES;
    a.eps = eps;
    const double inv = 1.0 / (double)head_dim;
    a.inv_dim = make_float2((float)inv, (float)(inv - (double)(float)inv));
    a.partial = nullptr;
    return Q4Q_OK;
}

}  // namespace

unsigned int rope_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_rope_status, &z, sizeof(z));
    return v;
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_rope_table(float* table, int64_t n_pos, int rot, double base, q4q_stream_t stream) {
    if (rot <= 0 || rot % 16 || rot > 256 || n_pos < 0 || n_pos >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (!(base > 0.0)) return Q4Q_ERR_ARG;
    if (n_pos == 0) return Q4Q_OK;
    if (!table) return Q4Q_ERR_NULL;
    if (!aligned(table, 16)) return Q4Q_ERR_ALIGN;
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    const int grid = (int)std::min<int64_t>((n_pos * (rot / 2) + THREADS - 1) / THREADS, (int64_t)info.sm_count * 16);
    rope_table_kernel<<<grid, THREADS, 0, (cudaStream_t)stream>>>(table, n_pos, rot, base);
    return launch_status();
}

extern "C" q4q_status q4q_qk_norm_rope(const void* q, int64_t q_stride, int n_q_heads, const void* k, int64_t k_stride, int n_k_heads, int type,
                                       int64_t head_dim, int64_t n_tokens, const float* q_weight, const float* k_weight, float eps,
                                       const float* table, int64_t n_pos, int rot, int mode, const int32_t* pos, void* q_dst, void* k_dst,
                                       q4q_stream_t stream) {
    RopeArgs a{};
    a.side[0] = {q, nullptr, q_weight, q_dst, q_stride, n_q_heads, 0, 0};
    a.side[1] = {k, nullptr, k_weight, k_dst, k_stride, n_k_heads, 0, 0};
    bool empty;
    q4q_status st = check(a, type, head_dim, n_tokens, table, n_pos, rot, mode, pos, eps, false, empty);
    if (st != Q4Q_OK || empty) return st;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    int blocks;
    return run(a, type, false, (cudaStream_t)stream, info, blocks);
}

extern "C" q4q_status q4q_qk_norm_rope_back_workspace_size(int64_t head_dim, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    if (!kv_dim_ok(head_dim)) return Q4Q_ERR_SHAPE;
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    *bytes = sizeof(float) * 2 * (size_t)head_dim * back_blocks(info);
    return Q4Q_OK;
}

extern "C" q4q_status q4q_qk_norm_rope_back(const void* d_q_dst, const void* d_k_dst, const void* q, int64_t q_stride, int n_q_heads, const void* k,
                                            int64_t k_stride, int n_k_heads, int type, int64_t head_dim, int64_t n_tokens, const float* q_weight,
                                            const float* k_weight, float eps, const float* table, int64_t n_pos, int rot, int mode,
                                            const int32_t* pos, void* d_q, void* d_k, float* d_q_weight, float* d_k_weight, void* workspace,
                                            size_t workspace_bytes, q4q_stream_t stream_) {
    RopeArgs a{};
    a.side[0] = {q, d_q_dst, q_weight, d_q, q_stride, n_q_heads, 0, 0};
    a.side[1] = {k, d_k_dst, k_weight, d_k, k_stride, n_k_heads, 0, 0};
    bool empty;
    q4q_status st = check(a, type, head_dim, n_tokens, table, n_pos, rot, mode, pos, eps, true, empty);
    if (st != Q4Q_OK) return st;
    if (!aligned(d_q_weight, 4) || !aligned(d_k_weight, 4)) return Q4Q_ERR_ALIGN;
    // a weight's gradient is written where the weight is given
    float* dwq = q_weight ? d_q_weight : nullptr;
    float* dwk = k_weight ? d_k_weight : nullptr;
    if ((q_weight && !d_q_weight) || (k_weight && !d_k_weight)) return Q4Q_ERR_NULL;
    cudaStream_t stream = (cudaStream_t)stream_;
    if (empty) {
        // sums over nothing
        if (dwq && cudaMemsetAsync(dwq, 0, sizeof(float) * head_dim, stream) != cudaSuccess) return cudaGetLastError(), Q4Q_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, sizeof(float) * head_dim, stream) != cudaSuccess) return cudaGetLastError(), Q4Q_ERR_CUDA;
        return Q4Q_OK;
    }
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    if (dwq || dwk) {
        size_t need = 0;
        if ((st = q4q_qk_norm_rope_back_workspace_size(head_dim, &need)) != Q4Q_OK) return st;
        if (!workspace) return Q4Q_ERR_NULL;
        if (!aligned(workspace, 256)) return Q4Q_ERR_ALIGN;
        if (workspace_bytes < need) return Q4Q_ERR_WORKSPACE;
        a.partial = static_cast<float*>(workspace);
    }
    int blocks;
    if ((st = run(a, type, true, stream, info, blocks)) != Q4Q_OK || !a.partial) return st;
    return launch(weight_sum_kernel, (2 * a.dim + WARPS - 1) / WARPS, 0, stream, (const float*)a.partial, blocks, a.dim, dwq, dwk);
}
