// q4q_mxfp4.cu -- MXFP4 matrices: the encoder (q4q_quantize_mxfp4), the row gather
// (q4q_get_rows_mxfp4) and the activation encoder of the MXFP4 products.
//
// All three are bound by HBM (the encoder reads 4 bytes and writes 0.53 per fp32 value,
// the gather the reverse).  A warp takes 256 consecutive columns of one row: 8 values a
// lane in one or two 16-byte loads, four lanes a block, one 128-byte line of codes.
#include <algorithm>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_mxfp4_status = 0;

constexpr int THREADS = 256;

// rows_pad = rows rounded up to 128: the scale bytes past the matrix are written as 0
template <typename T>
__global__ void __launch_bounds__(THREADS)
encode_kernel(const T* __restrict__ src, bool vec, uint8_t* __restrict__ dst, int K, int64_t rows, int64_t rows_pad,
              int64_t nmats, int64_t mat_stride, int64_t code_bytes) {
    const int lane = threadIdx.x & 31;
    const int segs = (K + MX_KP - 1) / MX_KP, nkc = 2 * segs;
    const int64_t per_mat = rows_pad * segs, total = per_mat * nmats;
    for (int64_t u = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 5; u < total;
         u += (int64_t)gridDim.x * (THREADS / 32)) {
        const int64_t mat = u / per_mat, in = u - mat * per_mat;
        const int64_t r = in / segs;
        const int seg = (int)(in - r * segs);
        uint8_t* out = dst + mat * mat_stride;
        float v[8];
        const int col = seg * MX_KP + lane * 8;
        if (r < rows && col < K) {
            mx_load<T, 8>(src + (mat * rows + r) * K + col, vec, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        // the code plane ends on a 256-byte boundary: after an odd number of segments, one more of zeros
        const bool codes = r < rows || (r == rows && seg == 0 && (rows * segs) % 2 != 0);
        mx_encode_segment<false>(v, codes ? out + (r * segs + seg) * (MX_KP / 2) : nullptr,
                                 out + code_bytes + mx_scale_offset(r, 128, nkc, 2 * seg), MX_CHUNK);
    }
}

// The activations of a product: row i of the operand is row i of src (dense), or, for an
// expert's row, the row of its token.  Also zeroes the product's control words.
struct ActArgs {
    const void* src;
    uint8_t* codes;
    uint8_t* scales;
    unsigned int* ctrl;
    int64_t n_ctrl;
    int64_t n_src, n_rows;
    int64_t max_groups;
    const int32_t* first;      // null: dense
    const int32_t* slot;       // null: row i of src is row i
    int n_experts, top_k, K, bn;
    bool vec, pdl;
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(THREADS) acts_kernel(const ActArgs a) {
    extern __shared__ int seg_smem[];
    __shared__ int tmp[33];
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.pdl) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.n_ctrl; i += (int64_t)gridDim.x * THREADS)
        a.ctrl[i] = 0u;
    int* start = seg_smem;
    int* base = seg_smem + a.n_experts + 1;
    if (a.first) mx_segments(a.first, a.n_experts, a.n_rows, a.bn, a.max_groups, start, base, tmp);
    const int segs = (a.K + MX_KP - 1) / MX_KP, nkc = 2 * segs;
    constexpr int SEG_BYTES = E4M3 ? MX_KP : MX_KP / 2;
    const int64_t total = a.n_rows * segs;
    for (int64_t u = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 5; u < total;
         u += (int64_t)gridDim.x * (THREADS / 32)) {
        const int64_t r = total < (1ll << 32) ? (int64_t)((uint32_t)u / (uint32_t)segs) : u / segs;
        const int seg = (int)(u - r * segs);
        int64_t from = r, to = r;
        if (a.first) {
            // the expert with start[e] <= r < start[e + 1]; empty experts share a start
            if (r >= start[a.n_experts] || r < start[0]) continue;
            const int e = mx_find(start, a.n_experts, (int)r);
            to = (int64_t)base[e] * a.bn + (r - start[e]);
            if (to >= (int64_t)base[e + 1] * a.bn) continue;
            if (a.slot) from = (int64_t)__ldg(a.slot + r) / a.top_k;
        }
        float v[8];
        const int col = seg * MX_KP + lane * 8;
        if (from >= 0 && from < a.n_src && col < a.K) {
            mx_load<T, 8>(static_cast<const T*>(a.src) + from * a.K + col, a.vec, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        mx_encode_segment<E4M3>(v, a.codes + (to * segs + seg) * SEG_BYTES,
                                a.scales + mx_scale_offset(to, a.bn, nkc, 2 * seg), mx_chunk_bytes(a.bn));
    }
}

// Row gather: 8 values a thread, two 16-byte streaming stores.
__global__ void __launch_bounds__(THREADS)
mx_get_rows_kernel(const uint8_t* __restrict__ table, int64_t code_bytes, int64_t nrows, int K,
                   const int32_t* __restrict__ ids, int64_t n, float* __restrict__ dst) {
    const int per_row = K / 8, segs = (K + MX_KP - 1) / MX_KP, nkc = 2 * segs;
    const int64_t total = n * per_row;
    for (int64_t g = blockIdx.x * (int64_t)THREADS + threadIdx.x; g < total; g += (int64_t)gridDim.x * THREADS) {
        const int64_t i = total < (1ll << 32) ? (int64_t)((uint32_t)g / (uint32_t)per_row) : g / per_row;
        const int c = (int)(g - i * per_row);
        const int64_t id = ids ? (int64_t)__ldg(ids + i) : i;
        float v[8];
        if (id < 0 || id >= nrows) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
            if (c == 0) record_error(&g_mxfp4_status, Q4Q_ERR_ARG);
        } else {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(table + id * (segs * (MX_KP / 2))) + c);
            const int b = c >> 2;
            const uint32_t sf = __ldg(table + code_bytes + mx_scale_offset(id, 128, nkc, b >> 2) + (b & 3));
            // 2^(sf - 127); sf = 0 is the subnormal 2^-127, 255 the format's NaN
            const float s = __uint_as_float(sf == 255 ? 0x7fffffffu : sf == 0 ? 0x00400000u : sf << 23);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const __half2_raw p = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w >> (8 * h)) & 0xffu), __NV_E2M1);
                v[2 * h] = __fmul_rn(__half2float(__half(__half_raw{p.x})), s);
                v[2 * h + 1] = __fmul_rn(__half2float(__half(__half_raw{p.y})), s);
            }
        }
        float4* o = reinterpret_cast<float4*>(dst + i * (int64_t)K + c * 8);
        __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
}

template <typename T>
q4q_status launch_acts_t(const ActArgs& a, bool e4m3, int grid, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pdl ? 1 : 0;
    const cudaError_t e = e4m3 ? cudaLaunchKernelEx(&cfg, acts_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, acts_kernel<T, false>, a);
    return e == cudaSuccess ? launch_status() : (cudaGetLastError(), Q4Q_ERR_CUDA);
}

}  // namespace

unsigned int mxfp4_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mxfp4_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_mxfp4_status, &z, sizeof(z));
    return v;
}

q4q_status mx_encode_acts(const MxActs& m, unsigned int* ctrl, int64_t n_ctrl, uint8_t* codes, uint8_t* scales, int bn,
                          int64_t max_groups, bool pdl, cudaStream_t stream, const DeviceInfo& info) {
    ActArgs a;
    a.src = m.src;
    a.codes = codes;
    a.scales = scales;
    a.ctrl = ctrl;
    a.n_ctrl = n_ctrl;
    a.n_src = m.n_src;
    a.n_rows = m.n_rows;
    a.max_groups = max_groups;
    a.first = m.first;
    a.slot = m.slot;
    a.n_experts = m.first ? m.n_experts : 0;
    a.top_k = m.top_k;
    a.K = (int)m.K;
    a.bn = bn;
    a.vec = aligned(m.src, 16);
    a.pdl = pdl;
    const int64_t units = m.n_rows * ((m.K + MX_KP - 1) / MX_KP);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((units + THREADS / 32 - 1) / (THREADS / 32), (int64_t)info.sm_count * 8));
    const size_t smem = m.first ? 2 * (size_t)(m.n_experts + 1) * sizeof(int) : 0;
    switch (m.type) {
        case Q4Q_TYPE_F32: return launch_acts_t<float>(a, m.acts == Q4Q_ACTS_MXFP8, grid, smem, stream);
        case Q4Q_TYPE_F16: return launch_acts_t<__half>(a, m.acts == Q4Q_ACTS_MXFP8, grid, smem, stream);
        default: return launch_acts_t<__nv_bfloat16>(a, m.acts == Q4Q_ACTS_MXFP8, grid, smem, stream);
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
    const int64_t rows_pad = mx_up(nrows, 128), units = rows_pad * (mx_up(ncols, MX_KP) / MX_KP) * nmats;
    const int64_t codes = mx_code_bytes(ncols, nrows), stride = codes + mx_scale_bytes(ncols, nrows);
    const int grid = (int)std::min<int64_t>((units + THREADS / 32 - 1) / (THREADS / 32), (int64_t)info.sm_count * 8);
    const bool vec = aligned(src, 16);
    uint8_t* out = static_cast<uint8_t*>(dst);
    cudaStream_t stream = (cudaStream_t)stream_;
    switch (src_type) {
        case Q4Q_TYPE_F32:
            encode_kernel<float><<<grid, THREADS, 0, stream>>>(static_cast<const float*>(src), vec, out, (int)ncols, nrows, rows_pad, nmats, stride, codes);
            break;
        case Q4Q_TYPE_F16:
            encode_kernel<__half><<<grid, THREADS, 0, stream>>>(static_cast<const __half*>(src), vec, out, (int)ncols, nrows, rows_pad, nmats, stride, codes);
            break;
        default:
            encode_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(static_cast<const __nv_bfloat16*>(src), vec, out, (int)ncols, nrows, rows_pad, nmats, stride, codes);
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
    const int64_t items = n_ids * (ne00 / 8);
    const int grid = (int)std::min<int64_t>((items + THREADS - 1) / THREADS, (int64_t)info.sm_count * 16);
    mx_get_rows_kernel<<<grid, THREADS, 0, (cudaStream_t)stream>>>(static_cast<const uint8_t*>(src0), mx_code_bytes(ne00, ne01), ne01, (int)ne00, ids, n_ids, dst);
    return launch_status();
}
