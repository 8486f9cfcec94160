// q4q_mxfp4.cu -- MXFP4 matrices: the encoder (q4q_quantize_mxfp4), the row gather
// (q4q_get_rows_mxfp4) and the activation encoder of the MXFP4 products.
//
// All three are bound by HBM (the encoder reads 4 bytes and writes 0.53 per fp32 value,
// the gather the reverse).  A unit is a segment of 256 consecutive columns of one row: in the
// encoders 8 values a lane in one or two 16-byte loads, four lanes a block, one 128-byte line
// of codes; in the gather 4 values a lane twice, so that each of a warp's 16-byte stores is
// one piece of 512 bytes.  A warp takes UNITS units of a row at a time, their loads in flight
// together.  What keeps the encoders from HBM's rate is their instructions (about 150 a
// warp's segment of 256 values, 8 a lane): 14336 x 4096 fp32 in 54 us (4.9 TB/s), 50257 x 768
// bf16 in 24.7 (3.9 TB/s), activations 2048 x 14336 fp32 in 26 (5.6 TB/s); the gather of
// 50257 x 768 takes 26.3 (6.6 TB/s).
#include <algorithm>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_internal.h"
#include "q4q_mx_tc.cuh"

namespace q4q {
namespace {

__device__ unsigned int g_mxfp4_status = 0;

constexpr int THREADS = 256;

// Position of the gather's warp in a line of units: row u / segs and segment u % segs, advanced
// without a division.
struct Unit {
    int64_t row;
    int seg;
    __device__ __forceinline__ Unit(int64_t u, int segs, bool small) {
        row = small ? (int64_t)((uint32_t)u / (uint32_t)segs) : u / segs;
        seg = (int)(u - row * segs);
    }
    __device__ __forceinline__ void next(int segs) {
        if (++seg == segs) {
            seg = 0;
            ++row;
        }
    }
};

// A warp's `n` next segments of one row: where its lane's columns start, whether the last
// segment of the row is cut short for this lane.
template <typename T, int UNITS>
__device__ __forceinline__ void load_segments(MxRaw<T> (&v)[UNITS], const T* p, int n, bool short_end, bool vec, const T* anywhere) {
#pragma unroll
    for (int k = 0; k < UNITS; ++k) v[k].live = k < n && !(short_end && k == n - 1);
    if (vec) {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) v[k].load16(v[k].live ? p + k * MX_KP : anywhere);
    } else {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) v[k].load(v[k].live ? p + k * MX_KP : anywhere, false);
    }
}

template <bool E4M3, typename T, int UNITS>
__device__ __forceinline__ void encode_segments(const MxRaw<T> (&v)[UNITS], uint8_t* codes, uint8_t* scales, int n, int chunk) {
#pragma unroll
    for (int k = 0; k < UNITS; ++k)
        if (k < n) mx_encode_segment<E4M3>(v[k], codes + k * (E4M3 ? MX_KP : MX_KP / 2), scales + 2 * k * chunk);
}

// Segments of an encoder's warp at a time: as many as keep its raw values in 16 registers, so that
// four blocks share an SM.
template <typename T>
constexpr int at_a_time = sizeof(T) == 4 ? 2 : 4;

// One matrix for each blockIdx.y (and every gridDim.y-th after it).
template <typename T, int UNITS>
__global__ void __launch_bounds__(THREADS, 4)
encode_kernel(const T* __restrict__ src, bool vec, uint8_t* __restrict__ dst, int K, int64_t rows, int64_t nmats,
              int64_t mat_stride, int64_t code_bytes) {
    const int lane = threadIdx.x & 31;
    const int segs = (K + MX_KP - 1) / MX_KP, nkc = 2 * segs, last = K - (segs - 1) * MX_KP;
    const int per_row = (segs + UNITS - 1) / UNITS;
    const int64_t total = rows * per_row;
    const bool small = total < (1ll << 31);
    for (int64_t mat = blockIdx.y; mat < nmats; mat += gridDim.y) {
        const T* in = src + mat * rows * K;
        uint8_t* out = dst + mat * mat_stride;
        uint8_t* scales = out + code_bytes + (lane >> 4) * MX_CHUNK;
        for (int64_t g = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 5; g < total; g += (int64_t)gridDim.x * (THREADS / 32)) {
            const int64_t r = small ? (int64_t)((uint32_t)g / (uint32_t)per_row) : g / per_row;
            const int s0 = (int)(g - r * per_row) * UNITS, n = min(UNITS, segs - s0);
            MxRaw<T> v[UNITS];
            load_segments(v, in + r * K + s0 * MX_KP + lane * 8, n, s0 + n == segs && lane * 8 >= last, vec, in);
            encode_segments<false>(v, out + (r * segs + s0) * (MX_KP / 2) + lane * 4,
                                   scales + mx_scale_offset(r, 7, MX_CHUNK, nkc, 2 * s0), n, MX_CHUNK);
        }
        // what lies past the matrix: the code plane ends on a 256-byte boundary, the scales' last
        // row group has 128 rows
        if (blockIdx.x == 0) {
            if (rows * segs % 2 != 0 && threadIdx.x < 32) reinterpret_cast<uint32_t*>(out + rows * segs * (MX_KP / 2))[lane] = 0u;
            const int64_t pad = (mx_up(rows, 128) - rows) * nkc;
            for (int64_t i = threadIdx.x; i < pad; i += THREADS)
                *reinterpret_cast<uint32_t*>(out + code_bytes + mx_scale_offset(rows + i / nkc, 7, MX_CHUNK, nkc, (int)(i % nkc))) = 0u;
        }
    }
}

// The activations of a product: row i of the operand is row i of src (dense), or, for an
// expert's row, the row of its token.  Also zeroes the product's abort word.
struct ActArgs {
    const void* src;
    uint8_t* codes;
    uint8_t* scales;
    unsigned int* abort_word;
    int64_t n_src, n_rows;
    int64_t max_groups;
    const int32_t* first;      // null: dense
    const int32_t* slot;       // null: row i of src is row i
    int n_experts, top_k, K, bn, bn_log;
    bool vec, pdl;
};

template <typename T, bool E4M3, int UNITS>
__global__ void __launch_bounds__(THREADS, 4) acts_kernel(const ActArgs a) {
    extern __shared__ int seg_smem[];
    __shared__ int tmp[33];
    const int lane = threadIdx.x & 31;
    // The kernel is always launched with programmatic dependent launch, so that its start
    // overlaps the end of the work before it.  The product behind it may read weights at once
    // when it starts: that is after the work before this kernel, unless the caller says that
    // none of it writes weights (Q4Q_MUL_MAT_PDL).
    if (a.pdl) pdl_trigger();
    pdl_wait();
    if (!a.pdl) pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.abort_word = 0u;
    const int segs = (a.K + MX_KP - 1) / MX_KP, nkc = 2 * segs, chunk = mx_chunk_bytes(a.bn), last = a.K - (segs - 1) * MX_KP;
    constexpr int LANE_BYTES = E4M3 ? 8 : 4;
    const T* src = static_cast<const T*>(a.src);
    uint8_t* scales = a.scales + (lane >> 4) * chunk;
    const int per_row = (segs + UNITS - 1) / UNITS;
    const int64_t total = a.n_rows * per_row, step = (int64_t)gridDim.x * (THREADS / 32);
    const bool small = total < (1ll << 31);
    MxRaw<T> v[UNITS];
    int64_t r = 0;
    int s0 = 0, n = 0;
    // the loads of group g: segments s0 .. s0 + n - 1 of sorted row r, by way of its slot
    auto load = [&](int64_t g) {
        r = small ? (int64_t)((uint32_t)g / (uint32_t)per_row) : g / per_row;
        s0 = (int)(g - r * per_row) * UNITS;
        n = min(UNITS, segs - s0);
        const int64_t row = a.slot ? (int64_t)((uint32_t)__ldg(a.slot + r) / (uint32_t)a.top_k) : r;
        if (row < a.n_src) {
            load_segments(v, src + row * a.K + s0 * MX_KP + lane * 8, n, s0 + n == segs && lane * 8 >= last, a.vec, src);
        } else {
#pragma unroll
            for (int k = 0; k < UNITS; ++k) v[k] = MxRaw<T>{};
        }
    };
    int64_t g = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 5;
    if (g < total) load(g);
    // where the rows go is worked out while the first loads are in flight
    int* start = seg_smem;
    int* base = seg_smem + a.n_experts + 1;
    if (a.first) mx_segments(a.first, a.n_experts, a.n_rows, a.bn, a.max_groups, start, base, tmp);
    // the operand row of sorted row r; negative: none
    auto place = [&](int64_t r) -> int64_t {
        if (!a.first) return r;
        // the expert with start[e] <= r < start[e + 1]; empty experts share a start
        if (r >= start[a.n_experts] || r < start[0]) return -1;
        const int e = mx_find(start, a.n_experts, (int)r);
        const int64_t to = (int64_t)base[e] * a.bn + (r - start[e]);
        return to < (int64_t)base[e + 1] * a.bn ? to : -1;
    };
    while (g < total) {
        const int64_t to = place(r);
        if (to >= 0)
            encode_segments<E4M3>(v, a.codes + ((to * segs + s0) * 32 + lane) * LANE_BYTES,
                                  scales + mx_scale_offset(to, a.bn_log, chunk, nkc, 2 * s0), n, chunk);
        g += step;
        if (g < total) load(g);
    }
}

template <int UNITS>
__global__ void __launch_bounds__(THREADS)
mx_get_rows_kernel(const uint8_t* __restrict__ table, int64_t code_bytes, int64_t nrows, int K,
                   const int32_t* __restrict__ ids, int64_t n, float* __restrict__ dst) {
    const int lane = threadIdx.x & 31;
    const int segs = (K + MX_KP - 1) / MX_KP, nkc = 2 * segs;
    const int64_t total = n * segs;
    const bool small = total < (1ll << 31);
    for (int64_t u0 = (((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 5) * UNITS; u0 < total;
         u0 += (int64_t)gridDim.x * (THREADS / 32) * UNITS) {
        const Unit first(u0, segs, small);
        uint32_t code[UNITS][2], scale[UNITS][2];
        bool known[UNITS];
        Unit at = first;
#pragma unroll
        for (int k = 0; k < UNITS; ++k, at.next(segs)) {
            const bool in = u0 + k < total;
            int64_t id = in ? (ids ? (int64_t)__ldg(ids + at.row) : at.row) : 0;
            known[k] = id >= 0 && id < nrows;
            if (!known[k]) {
                id = 0;
                if (lane == 0 && at.seg == 0 && in) record_error(&g_mxfp4_status, Q4Q_ERR_ARG);
            }
            // values 4 lane .. 4 lane + 3 of either half; the planes cover the padded columns
            const uint16_t* c = reinterpret_cast<const uint16_t*>(table + (id * segs + at.seg) * (MX_KP / 2)) + lane;
            const uint8_t* sc = table + code_bytes + mx_scale_offset(id, 7, MX_CHUNK, nkc, 2 * at.seg) + (lane >> 3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                code[k][h] = nrows > 0 ? __ldg(c + 32 * h) : 0;
                scale[k][h] = nrows > 0 ? __ldg(sc + h * MX_CHUNK) : 0;
            }
        }
        at = first;
#pragma unroll
        for (int k = 0; k < UNITS; ++k, at.next(segs)) {
            if (u0 + k >= total) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = at.seg * MX_KP + h * 128 + lane * 4;
                if (col >= K) continue;
                // 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 the format's NaN
                const uint32_t sf = scale[k][h];
                const float s = __uint_as_float(sf == 255 ? 0x7fffffffu : sf == 0 ? 0x00400000u : sf << 23);
                float v[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2_raw p = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((code[k][h] >> (8 * j)) & 0xffu), __NV_E2M1);
                    v[2 * j] = known[k] ? __fmul_rn(__half2float(__half(__half_raw{p.x})), s) : 0.0f;
                    v[2 * j + 1] = known[k] ? __fmul_rn(__half2float(__half(__half_raw{p.y})), s) : 0.0f;
                }
                __stcs(reinterpret_cast<float4*>(dst + at.row * (int64_t)K + col), make_float4(v[0], v[1], v[2], v[3]));
            }
        }
    }
}

// Units a warp takes at a time: several where one each would take more than one round of the
// SMs' 32 resident warps (2068 rows of 1504 routed to 32 experts: 8.5 us with one, 5.8 with 4)
bool many(int64_t units, const DeviceInfo& info) { return units > (int64_t)info.sm_count * 32; }

int grid_of(int64_t units, int units_at_a_time, const DeviceInfo& info) {
    const int64_t warps = (units + units_at_a_time - 1) / units_at_a_time;
    return (int)std::max<int64_t>(1, std::min<int64_t>((warps + THREADS / 32 - 1) / (THREADS / 32), (int64_t)info.sm_count * 8));
}

constexpr int AT_A_TIME = 4;      // units of the row gather's warp

template <typename T, bool E4M3>
q4q_status launch_acts_t(const ActArgs& a, cudaStream_t stream, const DeviceInfo& info) {
    constexpr int MANY = at_a_time<T>;
    const int64_t units = a.n_rows * ((a.K + MX_KP - 1) / MX_KP);
    const bool several = many(units, info);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid_of(units, several ? MANY : 1, info));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = a.first ? 2 * (size_t)(a.n_experts + 1) * sizeof(int) : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = several ? cudaLaunchKernelEx(&cfg, acts_kernel<T, E4M3, MANY>, a) : cudaLaunchKernelEx(&cfg, acts_kernel<T, E4M3, 1>, a);
    return e == cudaSuccess ? launch_status() : (cudaGetLastError(), Q4Q_ERR_CUDA);
}

template <typename T>
void launch_encode(const void* src, uint8_t* out, int64_t ncols, int64_t nrows, int64_t nmats, cudaStream_t stream, const DeviceInfo& info) {
    constexpr int MANY = at_a_time<T>;
    const int64_t units = nrows * (mx_up(ncols, MX_KP) / MX_KP);
    const int64_t codes = mx_code_bytes(ncols, nrows), stride = codes + mx_scale_bytes(ncols, nrows);
    const T* in = static_cast<const T*>(src);
    const bool vec = aligned(src, 16), several = many(units * nmats, info);
    const dim3 grid((unsigned)grid_of(units, several ? MANY : 1, info), (unsigned)std::min<int64_t>(nmats, 65535));
    if (several) encode_kernel<T, MANY><<<grid, THREADS, 0, stream>>>(in, vec, out, (int)ncols, nrows, nmats, stride, codes);
    else encode_kernel<T, 1><<<grid, THREADS, 0, stream>>>(in, vec, out, (int)ncols, nrows, nmats, stride, codes);
}

}  // namespace

unsigned int mxfp4_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mxfp4_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_mxfp4_status, &z, sizeof(z));
    return v;
}

q4q_status mx_encode_acts(const MxActs& m, unsigned int* abort_word, uint8_t* codes, uint8_t* scales, int bn,
                          int64_t max_groups, bool pdl, cudaStream_t stream, const DeviceInfo& info) {
    ActArgs a;
    a.src = m.src;
    a.codes = codes;
    a.scales = scales;
    a.abort_word = abort_word;
    a.n_src = m.n_src;
    a.n_rows = m.n_rows;
    a.max_groups = max_groups;
    a.first = m.first;
    a.slot = m.slot;
    a.n_experts = m.first ? m.n_experts : 0;
    a.top_k = m.top_k;
    a.K = (int)m.K;
    a.bn = bn;
    a.bn_log = 0;
    while ((1 << a.bn_log) < bn) ++a.bn_log;
    a.vec = aligned(m.src, 16);
    a.pdl = pdl;
    const bool e4m3 = m.acts == Q4Q_ACTS_MXFP8;
    switch (m.type) {
        case Q4Q_TYPE_F32: return e4m3 ? launch_acts_t<float, true>(a, stream, info) : launch_acts_t<float, false>(a, stream, info);
        case Q4Q_TYPE_F16: return e4m3 ? launch_acts_t<__half, true>(a, stream, info) : launch_acts_t<__half, false>(a, stream, info);
        default: return e4m3 ? launch_acts_t<__nv_bfloat16, true>(a, stream, info) : launch_acts_t<__nv_bfloat16, false>(a, stream, info);
    }
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_mxfp4_size(int64_t ne00, int64_t ne01, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    q4q_status st = check_mul_mat_shapes(ne00, ne01, ne00, 0);
    if (st != Q4Q_OK) return st;
    *bytes = (size_t)(mx_code_bytes(ne00, ne01) + mx_scale_bytes(ne00, ne01));
    return Q4Q_OK;
}

extern "C" q4q_status q4q_quantize_mxfp4(const void* src, int src_type, void* dst, int64_t ncols, int64_t nrows,
                                         int64_t nmats, q4q_stream_t stream_) {
    q4q_status st = check_mul_mat_shapes(ncols, nrows, ncols, 0);
    if (st != Q4Q_OK) return st;
    if (nmats < 0 || nmats >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (nrows > 0 && nmats > 0 && (ncols * nrows >= (1ll << 40) || nmats >= (1ll << 40) / (ncols * nrows))) return Q4Q_ERR_SHAPE;
    if (!mx_type_ok(src_type)) return Q4Q_ERR_ARG;
    if (nrows == 0 || nmats == 0) return Q4Q_OK;
    if (!src || !dst) return Q4Q_ERR_NULL;
    if (!aligned(src, mx_type_bytes(src_type)) || !aligned(dst, 256)) return Q4Q_ERR_ALIGN;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    uint8_t* out = static_cast<uint8_t*>(dst);
    cudaStream_t stream = (cudaStream_t)stream_;
    switch (src_type) {
        case Q4Q_TYPE_F32: launch_encode<float>(src, out, ncols, nrows, nmats, stream, info); break;
        case Q4Q_TYPE_F16: launch_encode<__half>(src, out, ncols, nrows, nmats, stream, info); break;
        default: launch_encode<__nv_bfloat16>(src, out, ncols, nrows, nmats, stream, info);
    }
    return launch_status();
}

extern "C" q4q_status q4q_get_rows_mxfp4(const void* src0, int64_t ne00, int64_t ne01, const int32_t* ids,
                                         int64_t n_ids, float* dst, q4q_stream_t stream) {
    q4q_status st = check_mul_mat_shapes(ne00, ne01, ne00, 0);
    if (st != Q4Q_OK) return st;
    if (n_ids < 0 || n_ids >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    if (!ids && n_ids > ne01) return Q4Q_ERR_SHAPE;
    if (n_ids == 0) return Q4Q_OK;
    if (!src0 || !dst) return Q4Q_ERR_NULL;
    if (!aligned(src0, 256) || !aligned(dst, 16) || (ids && !aligned(ids, 4))) return Q4Q_ERR_ALIGN;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    const int64_t units = n_ids * (mx_up(ne00, MX_KP) / MX_KP), codes = mx_code_bytes(ne00, ne01);
    const uint8_t* table = static_cast<const uint8_t*>(src0);
    if (many(units, info))
        mx_get_rows_kernel<AT_A_TIME><<<grid_of(units, AT_A_TIME, info), THREADS, 0, (cudaStream_t)stream>>>(table, codes, ne01, (int)ne00, ids, n_ids, dst);
    else
        mx_get_rows_kernel<1><<<grid_of(units, 1, info), THREADS, 0, (cudaStream_t)stream>>>(table, codes, ne01, (int)ne00, ids, n_ids, dst);
    return launch_status();
}
