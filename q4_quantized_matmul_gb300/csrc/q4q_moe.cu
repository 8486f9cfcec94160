// q4q_moe.cu -- tokens sorted by expert and back, with the gradients.
//
// A router gives each of n tokens top_k experts: slot s = t * top_k + j holds ids[s].  The
// sorted order lists the slots by expert, equal experts by slot; slots whose id is outside
// [0, n_experts) (choices that were dropped) come last and belong to no expert.
//   first[e]  the first sorted row of expert e, first[n_experts] the first dropped row
//   slot[r]   the slot of sorted row r;  row[s]  the sorted row of slot s
// With used(s) = row[s] < first[n_experts]:
//   gather        sorted[row[s]] = used(s) ? x[t] : 0
//   gather_back   dx[t] = sum_{j: used} dsorted[row[s]]
//   combine       y[t] = sum_{j: used} w[s] * rows[row[s]]
//   combine_back  drows[row[s]] = used(s) ? w[s] * dy[t] : 0
//                 dw[s] = used(s) ? sum_c dy[t][c] * rows[row[s]][c] : 0
// Sums are fp32 in the order of j (combine) or in a fixed order over the columns (dw), and
// are rounded once when stored; nothing is added by atomics, so results do not vary.
//
// The sort is a counting sort in one launch of one cluster of up to 8 CTAs: every warp
// counts a contiguous run of slots into its own histogram, prefix sums over warps, CTAs
// (distributed shared memory) and experts turn the counts into places, and the warp walks
// its run again; votes on the ids' bits give equal ids within a warp their order.  It is
// bound by the latency of these steps: 2.0 us for 2 choices, 4.8 for 2068, 8.5 for 32764
// (back to back).
//
// The row movers are bound by HBM and move 16 bytes a thread.  8191 tokens of 2048 bf16,
// top 4, calls back to back: gather 25.6 us (168 MB, 6.6 TB/s), combine_back 50.2 (302 MB, 6.0),
// combine and gather_back 30.7 each (168 MB, 5.5).  The order of the rows is not what holds those
// two back, for combine_back reads them in the same order.  It gives a warp a whole row, several
// pieces of 512 bytes in flight; combine gives a warp 512 bytes of each of a token's top_k rows,
// whose loads follow one another.  With that mapping kept, 16 loads of a thread in flight and
// rows looked up ahead changed nothing.
#include <algorithm>
#include <atomic>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_internal.h"
#include "q4q_mx_tc.cuh"

namespace q4q {
namespace {

// -------------------------------------------------------------------- sort --

constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_CLUSTER = 8;
constexpr int KEYS = 4;

// histograms [warps][bins], CTA totals, cluster totals and places [bins], scan scratch
__host__ __device__ constexpr size_t sort_smem(int warps, int bins) { return ((size_t)(warps + 3) * bins + 40) * 4; }

// The lanes with this lane's k (its low `bits` bits, k >= 0); one vote a bit, far quicker than
// match.any with 32 warps of an SM at it.
__device__ __forceinline__ uint32_t same_key(int k, int bits) {
    uint32_t peers = __ballot_sync(0xffffffffu, k >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint32_t ones = __ballot_sync(0xffffffffu, (k >> b) & 1);
        peers &= (k >> b) & 1 ? ones : ~ones;
    }
    return peers;
}

__global__ void __launch_bounds__(SORT_THREADS)
sort_kernel(const int32_t* ids, int n, int n_experts, int32_t* first,
            int32_t* slot, int32_t* row, int per_warp) {
    extern __shared__ int sm[];
    pdl_trigger();                                       // what follows may start up; it waits for this kernel's end
    pdl_wait();
    const int bins = n_experts + 1, warps = blockDim.x >> 5, bits = 32 - __clz(n_experts);
    int* hist = sm;
    int* total = hist + warps * bins;
    int* sums = total + bins;
    int* place = sums + bins;
    int* scan = place + bins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t rank, ctas;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    for (int i = tid; i < warps * bins; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int* mine = hist + warp * bins;
    const int64_t s0 = ((int64_t)rank * warps + warp) * per_warp;
    const int64_t s1 = min((int64_t)n, s0 + per_warp);
    auto key = [&](int64_t s) {
        const int id = s < s1 ? mx_ld(ids + s) : -1;
        return s < s1 ? ((unsigned)id < (unsigned)n_experts ? id : n_experts) : -1;
    };
    // a run's first KEYS steps stay in registers for the second walk
    int keys[KEYS];
    const int steps = (int)((max(s1 - s0, (int64_t)0) + 31) / 32);
#pragma unroll
    for (int i = 0; i < KEYS; ++i) keys[i] = i < steps ? key(s0 + 32 * i + lane) : -1;
    auto count = [&](int k) {
        const uint32_t peers = same_key(k, bits);
        if (k >= 0 && (__ffs(peers) - 1) == lane) mine[k] += __popc(peers);
        __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
        if (i < steps) count(keys[i]);
    for (int i = KEYS; i < steps; ++i) count(key(s0 + 32 * (int64_t)i + lane));
    __syncthreads();
    // what the CTA's warps before each one counted, and all of them: a thread a bin where there
    // are few warps, else a warp a bin
    if (warps <= 4) {
        for (int e = tid; e < bins; e += blockDim.x) {
            int sum = 0;
            for (int w = 0; w < warps; ++w) {
                const int c = hist[w * bins + e];
                hist[w * bins + e] = sum;
                sum += c;
            }
            total[e] = sum;
        }
    } else for (int e = warp; e < bins; e += warps) {
        const int c = lane < warps ? hist[lane * bins + e] : 0;
        int sum = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane < warps) hist[lane * bins + e] = sum - c;
        if (lane == 31) total[e] = sum;
    }
    __syncthreads();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    // rows of bin e in the CTAs before this one, and in all of them: the other CTAs' totals in
    // flight together
    int all = 0, before = 0;
    const int per = (bins + (int)blockDim.x - 1) / (int)blockDim.x;
    const int e0 = tid * per, e1 = min(e0 + per, bins);
    for (int e = e0; e < e1; ++e) {
        int v[SORT_MAX_CLUSTER];
#pragma unroll
        for (int c = 0; c < SORT_MAX_CLUSTER; ++c) {
            v[c] = 0;
            if (c < (int)ctas) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[c]) : "r"(mapa_shared(smem_u32(total + e), c)) : "memory");
        }
        int b = 0, a = 0;
#pragma unroll
        for (int c = 0; c < SORT_MAX_CLUSTER; ++c) {
            if (c < (int)rank) b += v[c];
            a += v[c];
        }
        place[e] = b;
        sums[e] = a;
        all += a;
    }
    int inc = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    before = inc - all;
    if (e0 < bins)
        for (int w = 0; w < warp; ++w) before += scan[w];
    for (int e = e0; e < e1; ++e) {
        if (rank == 0) first[e] = before;
        place[e] += before;
        before += sums[e];
    }
    __syncthreads();
    auto put = [&](int i, int k) {
        const int64_t s = s0 + 32 * (int64_t)i + lane;
        const uint32_t peers = same_key(k, bits);
        int at = 0;
        if (k >= 0) at = mine[k] + place[k] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (k >= 0) {
            if ((__ffs(peers) - 1) == lane) mine[k] += __popc(peers);
            slot[at] = (int32_t)s;
            row[s] = at;
        }
        __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
        if (i < steps) put(i, keys[i]);
    for (int i = KEYS; i < steps; ++i) put(i, key(s0 + 32 * (int64_t)i + lane));
    // no CTA leaves while another may still read its totals
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
}

// -------------------------------------------------------------- row movers --

constexpr int THREADS = 256;

template <typename T, int V>
struct Vec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ldv(const T* p) {
    if constexpr (V * sizeof(T) == 16) {
        const uint4 u = mx_ld(reinterpret_cast<const uint4*>(p));
        return *reinterpret_cast<const Vec<T, V>*>(&u);
    } else {
        Vec<T, V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = mx_ld(p + i);
        return r;
    }
}

template <typename T, int V>
__device__ __forceinline__ void stv(T* p, const Vec<T, V>& r) {
    if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
    else
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = r.v[i];
}

struct Rows {
    int64_t n_tokens;
    int top_k, ne0, per_row;        // per_row: vectors of a row
    int n_experts;
    const int32_t* first;
    const int32_t* row;
};

// number of rows that belong to an expert, never more than there are
__device__ __forceinline__ int64_t kept_rows(const Rows& g) {
    return min((int64_t)mx_ld(g.first + g.n_experts), g.n_tokens * g.top_k);
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gather_kernel(const T* x, T* out, const Rows g) {
    pdl_trigger();
    pdl_wait();
    const int64_t kept = kept_rows(g), slots = g.n_tokens * g.top_k, total = g.n_tokens * g.per_row;
    for (int64_t i = blockIdx.x * (int64_t)THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t t = total < (1ll << 32) ? (int64_t)((uint32_t)i / (uint32_t)g.per_row) : i / g.per_row;
        const int64_t c = (i - t * g.per_row) * V;
        const Vec<T, V> v = ldv<T, V>(x + t * g.ne0 + c);
        Vec<T, V> zero;
#pragma unroll
        for (int k = 0; k < V; ++k) zero.v[k] = mx_from_f32<T>(0.0f);
        for (int j = 0; j < g.top_k; ++j) {
            const int64_t r = mx_ld(g.row + t * g.top_k + j);
            if (r >= 0 && r < slots) stv<T, V>(out + r * g.ne0 + c, r < kept ? v : zero);
        }
    }
}

// y[t] = sum_j w * rows[row]; without weights the gradient of the gather
template <typename T, int V>
__global__ void __launch_bounds__(THREADS)
combine_kernel(const T* rows, const float* w, T* y, const Rows g) {
    pdl_trigger();
    pdl_wait();
    const int64_t kept = kept_rows(g), total = g.n_tokens * g.per_row;
    for (int64_t i = blockIdx.x * (int64_t)THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t t = total < (1ll << 32) ? (int64_t)((uint32_t)i / (uint32_t)g.per_row) : i / g.per_row;
        const int64_t c = (i - t * g.per_row) * V;
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        for (int j = 0; j < g.top_k; ++j) {
            const int64_t r = mx_ld(g.row + t * g.top_k + j);
            if (r < 0 || r >= kept) continue;
            const float f = w ? mx_ld(w + t * g.top_k + j) : 1.0f;
            const Vec<T, V> v = ldv<T, V>(rows + r * g.ne0 + c);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = __fmaf_rn(f, mx_to_f32(v.v[k]), acc[k]);
        }
        Vec<T, V> o;
#pragma unroll
        for (int k = 0; k < V; ++k) o.v[k] = mx_from_f32<T>(acc[k]);
        stv<T, V>(y + t * g.ne0 + c, o);
    }
}

// a warp per slot: drows and the dot product for dw
template <typename T, int V>
__global__ void __launch_bounds__(THREADS)
combine_back_kernel(const T* dy, const T* rows, const float* w,
                    T* drows, float* dw, const Rows g) {
    pdl_trigger();
    pdl_wait();
    const int64_t kept = kept_rows(g), slots = g.n_tokens * g.top_k;
    const int lane = threadIdx.x & 31;
    for (int64_t s = (blockIdx.x * (int64_t)THREADS + threadIdx.x) >> 5; s < slots; s += (int64_t)gridDim.x * (THREADS / 32)) {
        const int64_t t = s / g.top_k, r = mx_ld(g.row + s);
        if (r < 0 || r >= slots) continue;
        const bool used = r < kept;
        const float f = used ? mx_ld(w + s) : 0.0f;
        float dot = 0.0f;
#pragma unroll 4
        for (int v = lane; v < g.per_row; v += 32) {
            const int64_t c = (int64_t)v * V;
            Vec<T, V> o;
            if (used) {
                const Vec<T, V> a = ldv<T, V>(dy + t * g.ne0 + c), b = ldv<T, V>(rows + r * g.ne0 + c);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = mx_to_f32(a.v[k]);
                    dot = __fmaf_rn(d, mx_to_f32(b.v[k]), dot);
                    o.v[k] = mx_from_f32<T>(__fmul_rn(f, d));
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) o.v[k] = mx_from_f32<T>(0.0f);
            }
            stv<T, V>(drows + r * g.ne0 + c, o);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (lane == 0) dw[s] = used ? dot : 0.0f;
    }
}

// -------------------------------------------------------------------- host --

q4q_status check_rows(int type, int64_t ne0, int64_t n_tokens, int top_k, int n_experts) {
    if (!mx_type_ok(type) || top_k < 1 || n_experts < 1 || n_experts > MX_MAX_EXPERTS) return Q4Q_ERR_ARG;
    if (ne0 <= 0 || ne0 >= (1 << 20) || n_tokens < 0 || n_tokens * (int64_t)top_k >= (1ll << 31) || n_tokens >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    return Q4Q_OK;
}

enum Mover { GATHER, COMBINE, COMBINE_BACK };

struct Buffers {
    const void *a, *b;
    const float* w;
    void* out;
    float* dw;
};

template <typename T, int V>
void launch_mover_v(Mover what, const Buffers& m, Rows g, const DeviceInfo& info, cudaStream_t stream) {
    g.per_row = g.ne0 / V;
    const int64_t items = what == COMBINE_BACK ? g.n_tokens * g.top_k * 32 : g.n_tokens * g.per_row;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((items + THREADS - 1) / THREADS, (int64_t)info.sm_count * 16));
    const T *a = static_cast<const T*>(m.a), *b = static_cast<const T*>(m.b);
    T* out = static_cast<T*>(m.out);
    // programmatic dependent launch: every kernel here waits for the work before it first thing,
    // and its own start overlaps that work's end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // a launch that fails is left for launch_status to report
    if (what == GATHER) (void)cudaLaunchKernelEx(&cfg, gather_kernel<T, V>, a, out, g);
    else if (what == COMBINE) (void)cudaLaunchKernelEx(&cfg, combine_kernel<T, V>, a, m.w, out, g);
    else (void)cudaLaunchKernelEx(&cfg, combine_back_kernel<T, V>, a, b, m.w, out, m.dw, g);
}

template <typename T>
void launch_mover_t(Mover what, const Buffers& m, const Rows& g, const DeviceInfo& info, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    // 16 bytes a thread where every row starts on a 16-byte boundary, else one element
    const bool vec = g.ne0 % V == 0 && aligned(m.a, 16) && aligned(m.out, 16) && (!m.b || aligned(m.b, 16));
    if (vec) launch_mover_v<T, V>(what, m, g, info, stream);
    else launch_mover_v<T, 1>(what, m, g, info, stream);
}

q4q_status run_mover(Mover what, const Buffers& m, int type, int64_t ne0, int64_t n_tokens, int top_k, const int32_t* first,
                     int n_experts, const int32_t* row, cudaStream_t stream) {
    q4q_status st = check_rows(type, ne0, n_tokens, top_k, n_experts);
    if (st != Q4Q_OK) return st;
    if (n_tokens == 0) return Q4Q_OK;
    if (!m.a || !m.out || !first || !row || (what == COMBINE_BACK && (!m.b || !m.w || !m.dw))) return Q4Q_ERR_NULL;
    const size_t es = mx_type_bytes(type);
    if (!aligned(m.a, es) || !aligned(m.b, es) || !aligned(m.out, es) || !aligned(m.w, 4) || !aligned(m.dw, 4) || !aligned(first, 4) || !aligned(row, 4))
        return Q4Q_ERR_ALIGN;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    const Rows g{n_tokens, top_k, (int)ne0, 0, n_experts, first, row};
    switch (type) {
        case Q4Q_TYPE_F32: launch_mover_t<float>(what, m, g, info, stream); break;
        case Q4Q_TYPE_F16: launch_mover_t<__half>(what, m, g, info, stream); break;
        default: launch_mover_t<__nv_bfloat16>(what, m, g, info, stream);
    }
    return launch_status();
}

}  // namespace
}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_moe_sort(const int32_t* ids, int64_t n_tokens, int top_k, int n_experts, int32_t* first,
                                   int32_t* slot, int32_t* row, q4q_stream_t stream_) {
    q4q_status st = check_rows(Q4Q_TYPE_F32, 1, n_tokens, top_k, n_experts);
    if (st != Q4Q_OK) return st;
    if (!first || (n_tokens > 0 && (!ids || !slot || !row))) return Q4Q_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(first, 4) || !aligned(slot, 4) || !aligned(row, 4)) return Q4Q_ERR_ALIGN;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    if (info.device < 0 || info.device >= 64) return Q4Q_ERR_CUDA;
    cudaStream_t stream = (cudaStream_t)stream_;
    const int64_t n = n_tokens * top_k;
    // a warp takes at least 32 slots; more CTAs once every warp of one has KEYS times that
    const int64_t want = std::max<int64_t>(1, (n + 31) / 32);
    const int warps = (int)std::min<int64_t>(want, SORT_WARPS);
    int ctas = 1;
    while (ctas < SORT_MAX_CLUSTER && (int64_t)ctas * SORT_WARPS * KEYS < want) ctas *= 2;
    const int64_t per = (n + (int64_t)ctas * warps - 1) / ((int64_t)ctas * warps);
    const int per_warp = (int)mx_up(std::max<int64_t>(per, 1), 32);
    const size_t smem = sort_smem(warps, n_experts + 1);
    static std::atomic<int> configured[64];
    if (smem > 48 * 1024 && !configured[info.device].load()) {
        if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sort_smem(SORT_WARPS, MX_MAX_EXPERTS + 1)) != cudaSuccess)
            return (cudaGetLastError(), Q4Q_ERR_CUDA);
        configured[info.device].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, sort_kernel, ids, (int)n, n_experts, first, slot, row, per_warp) != cudaSuccess)
        return (cudaGetLastError(), Q4Q_ERR_CUDA);
    return launch_status();
}

extern "C" q4q_status q4q_moe_gather(const void* src, int type, int64_t ne0, int64_t n_tokens, int top_k, const int32_t* first,
                                     int n_experts, const int32_t* row, void* dst, q4q_stream_t stream) {
    return run_mover(GATHER, Buffers{src, nullptr, nullptr, dst, nullptr}, type, ne0, n_tokens, top_k, first, n_experts, row, (cudaStream_t)stream);
}

extern "C" q4q_status q4q_moe_gather_back(const void* d_dst, int type, int64_t ne0, int64_t n_tokens, int top_k,
                                          const int32_t* first, int n_experts, const int32_t* row, void* d_src,
                                          q4q_stream_t stream) {
    return run_mover(COMBINE, Buffers{d_dst, nullptr, nullptr, d_src, nullptr}, type, ne0, n_tokens, top_k, first, n_experts, row, (cudaStream_t)stream);
}

extern "C" q4q_status q4q_moe_combine(const void* rows, int type, int64_t ne0, int64_t n_tokens, int top_k, const int32_t* first,
                                      int n_experts, const int32_t* row, const float* weights, void* dst, q4q_stream_t stream) {
    if (n_tokens > 0 && !weights && check_rows(type, ne0, n_tokens, top_k, n_experts) == Q4Q_OK) return Q4Q_ERR_NULL;
    return run_mover(COMBINE, Buffers{rows, nullptr, weights, dst, nullptr}, type, ne0, n_tokens, top_k, first, n_experts, row, (cudaStream_t)stream);
}

extern "C" q4q_status q4q_moe_combine_back(const void* d_dst, const void* rows, int type, int64_t ne0, int64_t n_tokens,
                                           int top_k, const int32_t* first, int n_experts, const int32_t* row,
                                           const float* weights, void* d_rows, float* d_weights, q4q_stream_t stream) {
    return run_mover(COMBINE_BACK, Buffers{d_dst, rows, weights, d_rows, d_weights}, type, ne0, n_tokens, top_k, first, n_experts, row, (cudaStream_t)stream);
}
