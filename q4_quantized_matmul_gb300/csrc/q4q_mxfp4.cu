// q4q_mxfp4.cu -- MXFP4 matrices: the encoder (q4q_quantize_mxfp4), the row gather
// (q4q_get_rows_mxfp4) and the activation encoder of the MXFP4 products.
//
// All three are bound by HBM (the encoder reads 4 bytes and writes 0.53 per fp32 value,
// the gather the reverse).
//
// In the encoders a lane holds 64 bytes of a row, in two loads of a 32-byte sector each: a
// whole block of a 16-bit type, half a block of fp32.  Eight values a lane, four lanes a
// block and two loads that are one piece for the warp, were slower, by their instructions:
// 117 for each 256 bf16 values of which 50257 x 768 took 24.4 us; a lane's whole block has no
// shuffles, one scale for 32 values, its maximum two values at a time, and took 18.3.  With its
// start under the end of the call before it, 50257 x 768 bf16 take 15.7 us (6.2 TB/s) and
// 14336 x 4096 fp32 38.7 (6.9 TB/s).
//
// In the gather a unit is a segment of 256 columns of one row: 4 values a lane twice, so that
// each of a warp's 16-byte stores is one piece of 512 bytes, a warp's 4 units in flight
// together: 50257 x 768 in 29.1 us, 14336 x 4096 in 43.7 (6.0 and 6.1 TB/s, back to back).
#include <algorithm>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_internal.h"
#include "q4q_mx_tc.cuh"

namespace q4q {
namespace {

__device__ unsigned int g_mxfp4_status = 0;

constexpr int THREADS = 256;
// Blocks of the encoders on an SM.  The activation encoder, which has its place to find as well,
// spills with five: 512 x 4096 bf16 take a product 29.2 us with them, 28.2 with four.
constexpr int ENCODE_BLOCKS = 5, ACTS_BLOCKS = 4;

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

// Where a lane's piece of a matrix of padded rows is: the blocks of a matrix in the order of its
// code plane, LANES lanes a block.
template <typename T>
struct Piece {
    int64_t row;
    int block;             // of the row
    int col;               // its first column; K or more: padding
    __device__ __forceinline__ Piece(int64_t i, const MxDivisor& blocks, bool small) {
        const int64_t b = i / MxRaw<T>::LANES;
        row = small ? (int64_t)mx_divide((uint32_t)b, blocks) : b / blocks.d;
        block = (int)(b - row * blocks.d);
        col = block * 32 + (int)(i % MxRaw<T>::LANES) * MxRaw<T>::N;
    }
    // whether the lane writes the block's scale byte
    __device__ __forceinline__ bool first() const { return MxRaw<T>::LANES == 1 || col % 32 == 0; }
};

// One matrix for each blockIdx.y (and every gridDim.y-th after it).
template <typename T>
__global__ void __launch_bounds__(THREADS, ENCODE_BLOCKS)
encode_kernel(const T* src, int align, uint8_t* dst, int K, int64_t rows, int64_t nmats,
              int64_t mat_stride, int64_t code_bytes, const MxDivisor blocks) {
    pdl_trigger();
    pdl_wait();
    constexpr int WORDS = MxRaw<T>::N / 8;
    const int nkc = blocks.d / 4;
    const int64_t total = rows * blocks.d * MxRaw<T>::LANES;
    const bool small = rows * blocks.d < (1ll << 31);
    for (int64_t mat = blockIdx.y; mat < nmats; mat += gridDim.y) {
        const T* in = src + mat * rows * K;
        uint8_t* out = dst + mat * mat_stride;
        // (rounded up to whole warps)
        for (int64_t i = blockIdx.x * (int64_t)THREADS + threadIdx.x; (i & ~31ll) < total; i += (int64_t)gridDim.x * THREADS) {
            const Piece<T> at(i, blocks, small);
            MxRaw<T> raw;
            if (i < total && at.col < K) raw.load(in + at.row * K + at.col, align);
            else raw.clear();
            uint32_t w[WORDS];
            const uint32_t sf = mx_encode<false>(raw, w);
            if (i < total) {
                mx_put(out + i * (4 * WORDS), w);
                if (at.first()) out[code_bytes + mx_scale_offset(at.row, 7, MX_CHUNK, nkc, at.block >> 2) + (at.block & 3)] = (uint8_t)sf;
            }
        }
        // what lies past the matrix: the code plane ends on a 256-byte boundary, the scales' last
        // row group has 128 rows
        if (blockIdx.x == 0) {
            if (rows * (blocks.d / 8) % 2 != 0 && threadIdx.x < 32)
                reinterpret_cast<uint32_t*>(out + rows * blocks.d * 16)[threadIdx.x] = 0u;
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
    int n_experts, top_k, K, bn, bn_log, align;
    MxDivisor blocks;
    bool pdl;
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(THREADS, ACTS_BLOCKS) acts_kernel(const ActArgs a) {
    extern __shared__ int seg_smem[];
    __shared__ int tmp[33];
    // The product behind this kernel may read weights at once when it starts: that is after the
    // work before this kernel, unless the caller says that none of it writes weights
    // (Q4Q_MUL_MAT_PDL).
    if (a.pdl) pdl_trigger();
    pdl_wait();
    if (!a.pdl) pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.abort_word = 0u;
    constexpr int WORDS = MxRaw<T>::N / (E4M3 ? 4 : 8);
    const T* src = static_cast<const T*>(a.src);
    const int nkc = a.blocks.d / 4, chunk = mx_chunk_bytes(a.bn);
    const int64_t total = a.n_rows * a.blocks.d * MxRaw<T>::LANES, step = (int64_t)gridDim.x * THREADS;
    const bool small = a.n_rows * a.blocks.d < (1ll << 31);
    MxRaw<T> raw;
    // the lane's piece of sorted row `row`, by way of its slot
    auto load = [&](const Piece<T>& at, bool in) {
        int64_t from = at.row;
        if (in && a.slot) from = (uint32_t)mx_ld(a.slot + at.row) / (uint32_t)a.top_k;
        if (in && at.col < a.K && from < a.n_src) raw.load(src + from * a.K + at.col, a.align);
        else raw.clear();
    };
    int64_t i = blockIdx.x * (int64_t)THREADS + threadIdx.x;
    if ((i & ~31ll) < total) load(Piece<T>(i, a.blocks, small), i < total);
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
    while ((i & ~31ll) < total) {
        const Piece<T> at(i, a.blocks, small);
        uint32_t w[WORDS];
        const uint32_t sf = mx_encode<E4M3>(raw, w);
        const int64_t to = i < total ? place(at.row) : -1;
        if (to >= 0) {
            mx_put(a.codes + ((to * a.blocks.d + at.block) * MxRaw<T>::LANES + i % MxRaw<T>::LANES) * (4 * WORDS), w);
            if (at.first()) a.scales[mx_scale_offset(to, a.bn_log, chunk, nkc, at.block >> 2) + (at.block & 3)] = (uint8_t)sf;
        }
        i += step;
        if ((i & ~31ll) < total) load(Piece<T>(i, a.blocks, small), i < total);
    }
}

template <int UNITS>
__global__ void __launch_bounds__(THREADS)
mx_get_rows_kernel(const uint8_t* table, int64_t code_bytes, int64_t nrows, int K,
                   const int32_t* ids, int64_t n, float* dst) {
    pdl_trigger();
    pdl_wait();
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
            int64_t id = in ? (ids ? (int64_t)mx_ld(ids + at.row) : at.row) : 0;
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
                code[k][h] = nrows > 0 ? mx_ld(c + 32 * h) : 0;
                scale[k][h] = nrows > 0 ? mx_ld(sc + h * MX_CHUNK) : 0;
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

// Units a warp of the gather takes at a time: several where one each would take more than one
// round of 32 resident warps an SM
bool many(int64_t units, const DeviceInfo& info) { return units > (int64_t)info.sm_count * 32; }

int grid_of(int64_t units, int units_at_a_time, const DeviceInfo& info) {
    const int64_t warps = (units + units_at_a_time - 1) / units_at_a_time;
    return (int)std::max<int64_t>(1, std::min<int64_t>((warps + THREADS / 32 - 1) / (THREADS / 32), (int64_t)info.sm_count * 8));
}

constexpr int AT_A_TIME = 4;      // units of the row gather's warp

// blocks of an encoder with a lane for each of `lanes` pieces: one piece a lane up to 8 rounds of
// the SMs' blocks (1 or 2 rounds measured the same within 2%)
int encoder_grid(int64_t lanes, int blocks, const DeviceInfo& info) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((lanes + THREADS - 1) / THREADS, (int64_t)info.sm_count * 8 * blocks));
}

int alignment(const void* p) { return aligned(p, 32) ? 32 : aligned(p, 16) ? 16 : 1; }

// All kernels here are launched with programmatic dependent launch, so that their start overlaps
// the end of the work before them, for which they wait first thing (encode and row gather of
// 50257 x 768 bf16, one call after another: 53.7 us without, 46.5 with).
template <typename... Params, typename... Args>
q4q_status launch(void (*kernel)(Params...), dim3 grid, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
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

template <typename T, bool E4M3>
q4q_status launch_acts_t(const ActArgs& a, cudaStream_t stream, const DeviceInfo& info) {
    return launch(acts_kernel<T, E4M3>, dim3((unsigned)encoder_grid(a.n_rows * a.blocks.d * MxRaw<T>::LANES, ACTS_BLOCKS, info)),
                  a.first ? 2 * (size_t)(a.n_experts + 1) * sizeof(int) : 0, stream, a);
}

template <typename T>
q4q_status launch_encode(const void* src, uint8_t* out, int64_t ncols, int64_t nrows, int64_t nmats, cudaStream_t stream, const DeviceInfo& info) {
    const MxDivisor blocks = mx_divisor((uint32_t)(mx_up(ncols, MX_KP) / 32));
    const int64_t codes = mx_code_bytes(ncols, nrows), stride = codes + mx_scale_bytes(ncols, nrows);
    const dim3 grid((unsigned)encoder_grid(nrows * blocks.d * MxRaw<T>::LANES, ENCODE_BLOCKS, info), (unsigned)std::min<int64_t>(nmats, 65535));
    return launch(encode_kernel<T>, grid, 0, stream, static_cast<const T*>(src), alignment(src), out, (int)ncols, nrows, nmats, stride,
                  codes, blocks);
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
    a.align = alignment(m.src);
    a.blocks = mx_divisor((uint32_t)(mx_up(m.K, MX_KP) / 32));
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
        case Q4Q_TYPE_F32: return launch_encode<float>(src, out, ncols, nrows, nmats, stream, info);
        case Q4Q_TYPE_F16: return launch_encode<__half>(src, out, ncols, nrows, nmats, stream, info);
        default: return launch_encode<__nv_bfloat16>(src, out, ncols, nrows, nmats, stream, info);
    }
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
    const bool several = many(units, info);
    return launch(several ? mx_get_rows_kernel<AT_A_TIME> : mx_get_rows_kernel<1>, dim3((unsigned)grid_of(units, several ? AT_A_TIME : 1, info)), 0,
                  (cudaStream_t)stream, table, codes, ne01, (int)ne00, ids, n_ids, dst);
}
