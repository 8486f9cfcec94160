// q4q_mx.cuh -- what the MXFP4 kernels share: the element types, the block encoders
// and the layout of the operand planes.
//
// Microscaling (OCP MX 1.0): a block is 32 values along K with one E8M0 scale 2^e.
//   e = floor(log2(amax)) - emax   (emax = 2 for E2M1, 8 for E4M3), at least -127
//   element = round_to_nearest_even(x * 2^-e), saturated at 6 (E2M1) or 448 (E4M3)
// x * 2^-e is exact in fp32 (a power of two; for amax below 2^-125, where e stops at
// -127, the product still only grows), so the hardware conversions round x itself once.
// A block of zeros has scale byte 0 and codes 0; one that holds an infinity or a NaN
// has scale byte 255 (the format's NaN) and codes 0: all of its values are NaN.
//
// Planes.  Codes: row-major, rows of Kp elements (Kp = K rounded up to 256, zeros past
// K), two per byte for E2M1 (low nibble first), one per byte for E4M3.  Scales: for each
// 128 rows and 128 columns 512 bytes in the order in which tcgen05.cp takes scale factors
// into tensor memory: the byte of row r, block b is at (r % 32) * 16 + (r / 32 % 4) * 4 + b.
// A tile of `bn` rows (128 for weights, a token tile's for activations) has for each 128
// columns one chunk: its 512-byte pieces, or, up to 32 rows, only the 16 bn bytes in use.
// Chunks are ordered by row tile, then by column, so a tile's K range is one piece.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>

#include "q4q_common.cuh"

namespace q4q {

constexpr int MX_KP = 256;            // K is padded to this
constexpr int MX_CHUNK = 512;         // scale bytes of 128 rows x 128 columns
constexpr int MX_MAX_EXPERTS = 1024;

// bytes of a row tile's scales for 128 columns
__host__ __device__ constexpr int mx_chunk_bytes(int bn) { return bn <= 32 ? bn * 16 : bn <= 128 ? MX_CHUNK : bn / 128 * MX_CHUNK; }

__host__ __device__ __forceinline__ int64_t mx_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
__host__ __device__ __forceinline__ int64_t mx_code_bytes(int64_t ne00, int64_t ne01) {
    return mx_up(ne01 * (mx_up(ne00, MX_KP) / 2), 256);
}
__host__ __device__ __forceinline__ int64_t mx_scale_bytes(int64_t ne00, int64_t ne01) {
    return mx_up(ne01, 128) * (mx_up(ne00, MX_KP) / 32);
}

template <typename T>
__device__ __forceinline__ float mx_to_f32(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T mx_from_f32(float v);
template <>
__device__ __forceinline__ float mx_from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half mx_from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 mx_from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 8 values of T as they were loaded, looked at only when they are needed; `live`: not zeros
// (the same in the four lanes of a block).
template <typename T>
struct MxRaw {
    uint4 bits[sizeof(T) / 2];
    bool live;
    // `vec`: p is 16-byte aligned
    __device__ __forceinline__ void load(const T* __restrict__ p, bool vec) {
        if (vec) {
            load16(p);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) reinterpret_cast<T*>(bits)[k] = p[k];
        }
    }
    __device__ __forceinline__ void load16(const T* __restrict__ p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) bits[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = mx_to_f32(reinterpret_cast<const T*>(bits)[k]);
    }
};

// the largest magnitude of three, NaN if one is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Encode 8 values a lane, four neighbouring lanes a block (the whole converged warp calls
// it): the codes in w (8 bytes for E4M3, 4 for E2M1), the block's scale byte returned.
template <bool E4M3>
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], bool live, uint32_t (&w)[2]) {
    constexpr int EMAX = E4M3 ? 8 : 2;
    float m = max3_abs(v[0], v[1], v[2]);
    m = max3_abs(m, v[3], v[4]);
    m = max3_abs(m, v[5], v[6]);
    m = max3_abs(m, v[7], __shfl_xor_sync(0xffffffffu, max3_abs(m, v[7], v[7]), 1));
    m = max3_abs(m, m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int field = (int)(__float_as_uint(m) >> 23);             // 255: the block holds an infinity or a NaN
    const bool use = live && field != 255;
    int sf = max(field - EMAX, 0);                                 // e + 127; 0 also where amax is 0 or subnormal
    // 2^-e = 2^(127 - sf): 127 - sf is -126 .. 127 for finite blocks
    const float inv = __uint_as_float((uint32_t)(254 - sf) << 23);
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = __fmul_rn(v[k], inv);
    if constexpr (E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm("{\n\t.reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                "mov.b32 %0, {a, b};\n\t}"
                : "=r"(w[h]) : "f"(t[4 * h]), "f"(t[4 * h + 1]), "f"(t[4 * h + 2]), "f"(t[4 * h + 3]));
        w[0] = use ? w[0] : 0u;
        w[1] = use ? w[1] : 0u;
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(w[0]) : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
        w[0] = use ? w[0] : 0u;
        w[1] = 0u;
    }
    sf = use ? sf : live ? 255 : 0;
    return (uint32_t)sf;
}

// Encode 256 consecutive columns of one row: lane l of the (converged) warp holds columns
// 8l .. 8l+7.  Writes the lane's codes at `codes` and, from lanes 0 and 16, the four scale
// bytes of each half of the segment at `scales`.
template <bool E4M3, typename T>
__device__ __forceinline__ void mx_encode_segment(const MxRaw<T>& raw, uint8_t* codes, uint8_t* scales) {
    float v[8];
    raw.values(v);
    uint32_t w[2];
    uint32_t word = mx_encode8<E4M3>(v, raw.live, w);
    if constexpr (E4M3) *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(codes) = w[0];
    // the bytes of lanes l, l+4, l+8, l+12
    word |= __shfl_down_sync(0xffffffffu, word, 4) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
    if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(scales) = word;
}

// dst[i] = v, rounded to the type
__device__ __forceinline__ void mx_store(void* dst, int type, int64_t i, float v) {
    if (type == Q4Q_TYPE_F32) static_cast<float*>(dst)[i] = v;
    else if (type == Q4Q_TYPE_F16) static_cast<__half*>(dst)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16_rn(v);
}

// Offset of the scale word of row r for the 128 columns kc, in tiles of 2^bn_log rows whose
// chunks take `chunk` bytes.
__device__ __forceinline__ int64_t mx_scale_offset(int64_t r, int bn_log, int chunk, int nkc, int kc) {
    const int64_t tile = r >> bn_log;
    const int in = (int)r & ((1 << bn_log) - 1);
    return (tile * nkc + kc) * chunk + (in >> 7) * MX_CHUNK + (in & 31) * 16 + ((in >> 5) & 3) * 4;
}

// The experts' segments: rows start[e] .. start[e + 1] - 1 of the sorted order, at row
// base[e] * bn of the activation operand (every segment starts a new token tile).  Whatever
// `first` holds, no segment leaves [0, n_rows) and all of them together take at most
// max_groups token tiles.  All of the block's threads call it (a multiple of 32, at most
// 1024); `tmp` holds 33 words.
__device__ __forceinline__ void mx_segments(const int32_t* __restrict__ first, int n_experts, int64_t n_rows, int bn,
                                            int64_t max_groups, int* start, int* base, int* tmp) {
    const int per = (n_experts + (int)blockDim.x - 1) / (int)blockDim.x;
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, n_experts);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto at = [&](int e) { return (int)min(max((int64_t)__ldg(first + e), (int64_t)0), n_rows); };
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += (max(at(e + 1) - at(e), 0) + bn - 1) / bn;
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += tmp[w];
    for (int e = e0; e < e1; ++e) {
        start[e] = at(e);
        base[e] = (int)min((int64_t)before, max_groups);
        before += (max(at(e + 1) - at(e), 0) + bn - 1) / bn;
        if (e == n_experts - 1) {
            start[n_experts] = at(n_experts);
            base[n_experts] = (int)min((int64_t)before, max_groups);
        }
    }
    __syncthreads();
}

// The e with base[e] <= g < base[e + 1].
__device__ __forceinline__ int mx_find(const int* base, int n_experts, int g) {
    int lo = 0, hi = n_experts;                        // base[lo] <= g < base[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= g) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace q4q
