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
// A row takes D / 8 lanes, 8 values each; a warp takes a token's rows one after another, so that the
// token's cosines, sines and weights are loaded once and several rows are in flight.  Bound by HBM
// when there are many tokens, by the launch and two loads behind one another when there are few.
// dw is summed in registers over a warp's rows, then over the block's warps, and the blocks' sums by a
// second kernel in the order of the blocks: no atomics, results do not vary.
#include <algorithm>

#include "q4q_attn.cuh"
#include "q4q_mx_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_rope_status = 0;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int IN_FLIGHT = 4;       // row slots that a warp loads ahead
constexpr int BACK_IN_FLIGHT = 2;

struct Side {                      // the queries, or the keys
    const void* x;                 // [tokens][heads][D], rows of a token at `stride` elements
    const void* dy;
    const float* w;
    void* out;                     // [tokens][heads][D]: y, or dx
    int64_t stride;
    int heads;
};

struct RopeArgs {
    Side side[2];
    const float* table;
    const int32_t* pos;
    int64_t n_pos, n_tokens;
    int dim, rot, halves, align;
    float eps;
    float2 inv_dim;
    int per;                       // row slots of a work item (a warp holds 32 / LANES rows in one slot)
    int items;                     // work items of a token
    float* partial;                // backward: [blocks][2][D]
};

// The lane's row in slot `slot` of a token: which side and head; false past the last.
__device__ __forceinline__ bool row_of(const RopeArgs& a, int row, int& side, int& head) {
    side = row >= a.side[0].heads;
    head = side ? row - a.side[0].heads : row;
    return row < a.side[0].heads + a.side[1].heads;
}

__device__ __forceinline__ void load_weights(const Side& s, int at, float (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        const uint4 u = mx_ld(reinterpret_cast<const uint4*>(s.w + at + e));
        w[e] = __uint_as_float(u.x), w[e + 1] = __uint_as_float(u.y), w[e + 2] = __uint_as_float(u.z), w[e + 3] = __uint_as_float(u.w);
    }
}

// the token's angles; false where its position has none (its rows become zeros)
__device__ __forceinline__ bool angles(const RopeArgs& a, int64_t token, int at, Turn& turning) {
    turning.turns = false;
    if (!a.table) return true;
    const int p = mx_ld(a.pos + token);
    if (p < 0 || p >= a.n_pos) {
        if ((threadIdx.x & 31) == 0) record_error(&g_rope_status, Q4Q_ERR_ARG);
        return false;
    }
    turn_load(turning, a.table + (int64_t)p * a.rot, a.rot, a.halves, at);
    return true;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(RopeArgs a) {
    constexpr int ROWS = 32 / LANES;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, at = lane % LANES * 8;
    const bool used = at < a.dim;
    const int64_t items = a.n_tokens * a.items;
    for (int64_t item = blockIdx.x * (int64_t)WARPS + (threadIdx.x >> 5); item < items; item += (int64_t)gridDim.x * WARPS) {
        const int64_t token = item / a.items;
        const int first = (int)(item - token * a.items) * a.per;
        Turn turning;
        const bool known = angles(a, token, used ? at : a.rot, turning);
        for (int s0 = 0; s0 < a.per; s0 += IN_FLIGHT) {
            float v[IN_FLIGHT][8];
            int side[IN_FLIGHT], head[IN_FLIGHT];
            bool here[IN_FLIGHT];
#pragma unroll
            for (int i = 0; i < IN_FLIGHT; ++i) {
                here[i] = row_of(a, (first + s0 + i) * ROWS + lane / LANES, side[i], head[i]) && used && s0 + i < a.per;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
                if (here[i]) {
                    const Side& s = a.side[side[i]];
                    row_load(static_cast<const T*>(s.x) + token * s.stride + (int64_t)head[i] * a.dim + at, a.align, v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < IN_FLIGHT; ++i) {
                if (!__any_sync(0xffffffffu, here[i])) break;
                const float* w = a.side[side[i]].w;
                if (__any_sync(0xffffffffu, here[i] && w)) {
                    const float r = inverse_norm<LANES>(v[i], a.inv_dim, a.eps);
                    if (here[i] && w) {
                        float ww[8];
                        load_weights(a.side[side[i]], at, ww);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i][e] = __fmul_rn(__fmul_rn(v[i][e], r), ww[e]);
                    }
                }
                if (a.table) turn(v[i], turning, a.halves, at, a.rot);
                if (here[i]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = known ? v[i][e] : 0.0f;
                    const Side& s = a.side[side[i]];
                    row_store(static_cast<T*>(s.out) + (token * s.heads + head[i]) * (int64_t)a.dim + at, a.align, v[i]);
                }
            }
        }
    }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(THREADS) norm_rope_back_kernel(RopeArgs a) {
    constexpr int ROWS = 32 / LANES;
    extern __shared__ float sums[];            // [warps][2][D] of the rows of a warp's first LANES lanes
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % LANES * 8;
    const bool used = at < a.dim;
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
    const int64_t items = a.n_tokens * a.items;
    for (int64_t item = blockIdx.x * (int64_t)WARPS + warp; item < items; item += (int64_t)gridDim.x * WARPS) {
        const int64_t token = item / a.items;
        const int first = (int)(item - token * a.items) * a.per;
        Turn turning;
        const bool known = angles(a, token, used ? at : a.rot, turning);
        for (int s0 = 0; s0 < a.per; s0 += BACK_IN_FLIGHT) {
            float g[BACK_IN_FLIGHT][8], x[BACK_IN_FLIGHT][8];
            int side[BACK_IN_FLIGHT], head[BACK_IN_FLIGHT];
            bool here[BACK_IN_FLIGHT];
#pragma unroll
            for (int i = 0; i < BACK_IN_FLIGHT; ++i) {
                here[i] = row_of(a, (first + s0 + i) * ROWS + lane / LANES, side[i], head[i]) && used && s0 + i < a.per;
#pragma unroll
                for (int e = 0; e < 8; ++e) g[i][e] = x[i][e] = 0.0f;
                if (here[i] && known) {
                    const Side& s = a.side[side[i]];
                    row_load(static_cast<const T*>(s.dy) + (token * s.heads + head[i]) * (int64_t)a.dim + at, a.align, g[i]);
                    if (s.w) row_load(static_cast<const T*>(s.x) + token * s.stride + (int64_t)head[i] * a.dim + at, a.align, x[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < BACK_IN_FLIGHT; ++i) {
                if (!__any_sync(0xffffffffu, here[i])) break;
                if (a.table) turn(g[i], turning, a.halves, at, a.rot, true);
                const Side& s = a.side[side[i]];
                const bool norm = here[i] && s.w;
                if (__any_sync(0xffffffffu, norm)) {
                    const float r = inverse_norm<LANES>(x[i], a.inv_dim, a.eps);
                    float w[8], dot = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0.0f;
                    if (norm) load_weights(s, at, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[i][e] *= norm && known ? r : 0.0f;                          // xh
                        const float part = g[i][e] * x[i][e];
                        // selected, not indexed: the sums stay in registers
                        dw[0][e] += side[i] == 0 && norm ? part : 0.0f;
                        dw[1][e] += side[i] == 1 && norm ? part : 0.0f;
                        if (norm) g[i][e] *= w[e];
                        dot = fmaf(g[i][e], x[i][e], dot);
                    }
                    dot = row_sum<LANES>(dot);
                    const float mean = fmaf(dot, a.inv_dim.x, dot * a.inv_dim.y);
                    if (norm)
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[i][e] = r * (g[i][e] - x[i][e] * mean);
                }
                if (here[i]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[i][e] = known ? g[i][e] : 0.0f;
                    row_store(static_cast<T*>(s.out) + (token * s.heads + head[i]) * (int64_t)a.dim + at, a.align, g[i]);
                }
            }
        }
    }
    if (!a.partial) return;
    // the warp's rows, then the block's warps
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[q][e];
#pragma unroll
            for (int d = LANES; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            if (lane < LANES && used) sums[(warp * 2 + q) * a.dim + at + e] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sums[w * 2 * a.dim + i];
        a.partial[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
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

// Row slots of a work item.  A warp that takes several rows of a token loads its angles once, but few
// tokens should use all SMs: the most (of 1, 2, 4, 8, 16) that leaves each SM two blocks' warps of
// work items.
void plan(RopeArgs& a, int lanes, const DeviceInfo& info) {
    const int rows = a.side[0].heads + a.side[1].heads, slots = (rows + 32 / lanes - 1) / (32 / lanes);
    a.per = 1;
    while (a.per < 16 && a.per < slots && a.n_tokens * ((slots + 2 * a.per - 1) / (2 * a.per)) >= (int64_t)info.sm_count * 2 * WARPS) a.per *= 2;
    a.items = (slots + a.per - 1) / a.per;
}

int blocks_of(const RopeArgs& a, int per_sm, const DeviceInfo& info) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((a.n_tokens * a.items + WARPS - 1) / WARPS, (int64_t)info.sm_count * per_sm));
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

// blocks a backward call may run at most: its workspace has one row of sums for each
constexpr int BACK_BLOCKS_PER_SM = 3;

template <typename T, int LANES>
q4q_status run_t(RopeArgs& a, bool back, cudaStream_t stream, const DeviceInfo& info) {
    plan(a, LANES, info);
    if (!back) return launch(norm_rope_kernel<T, LANES>, blocks_of(a, 8, info), 0, stream, a);
    return launch(norm_rope_back_kernel<T, LANES>, blocks_of(a, BACK_BLOCKS_PER_SM, info),
                  a.partial ? sizeof(float) * WARPS * 2 * a.dim : 0, stream, a);
}

template <typename T>
q4q_status run_lanes(RopeArgs& a, bool back, cudaStream_t stream, const DeviceInfo& info) {
    switch (lanes_of(a.dim)) {
        case 8: return run_t<T, 8>(a, back, stream, info);
        case 16: return run_t<T, 16>(a, back, stream, info);
        default: return run_t<T, 32>(a, back, stream, info);
    }
}

q4q_status run(RopeArgs& a, int type, bool back, cudaStream_t stream, const DeviceInfo& info) {
    switch (type) {
        case Q4Q_TYPE_F32: return run_lanes<float>(a, back, stream, info);
        case Q4Q_TYPE_F16: return run_lanes<__half>(a, back, stream, info);
        default: return run_lanes<__nv_bfloat16>(a, back, stream, info);
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
    a.side[0] = {q, nullptr, q_weight, q_dst, q_stride, n_q_heads};
    a.side[1] = {k, nullptr, k_weight, k_dst, k_stride, n_k_heads};
    bool empty;
    q4q_status st = check(a, type, head_dim, n_tokens, table, n_pos, rot, mode, pos, eps, false, empty);
    if (st != Q4Q_OK || empty) return st;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    return run(a, type, false, (cudaStream_t)stream, info);
}

extern "C" q4q_status q4q_qk_norm_rope_back_workspace_size(int64_t head_dim, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    if (!kv_dim_ok(head_dim)) return Q4Q_ERR_SHAPE;
    DeviceInfo info;
    const q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    *bytes = sizeof(float) * 2 * (size_t)head_dim * BACK_BLOCKS_PER_SM * info.sm_count;
    return Q4Q_OK;
}

extern "C" q4q_status q4q_qk_norm_rope_back(const void* d_q_dst, const void* d_k_dst, const void* q, int64_t q_stride, int n_q_heads, const void* k,
                                            int64_t k_stride, int n_k_heads, int type, int64_t head_dim, int64_t n_tokens, const float* q_weight,
                                            const float* k_weight, float eps, const float* table, int64_t n_pos, int rot, int mode,
                                            const int32_t* pos, void* d_q, void* d_k, float* d_q_weight, float* d_k_weight, void* workspace,
                                            size_t workspace_bytes, q4q_stream_t stream_) {
    RopeArgs a{};
    a.side[0] = {q, d_q_dst, q_weight, d_q, q_stride, n_q_heads};
    a.side[1] = {k, d_k_dst, k_weight, d_k, k_stride, n_k_heads};
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
    if ((st = run(a, type, true, stream, info)) != Q4Q_OK || !a.partial) return st;
    return launch(weight_sum_kernel, (2 * a.dim + WARPS - 1) / WARPS, 0, stream, (const float*)a.partial, blocks_of(a, BACK_BLOCKS_PER_SM, info),
                  a.dim, dwq, dwk);
}
