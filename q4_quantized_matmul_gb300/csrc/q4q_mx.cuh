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

// A load of what the work before this kernel may have written, for kernels that start before that
// work ends and wait for it (griddepcontrol.wait).  It is a plain ld.global: the non-coherent form
// (ld.global.nc, which is also what __ldg and reads through const __restrict__ pointers become) is
// for memory that nothing writes while the kernel runs, and may be served by, or moved up to, a time
// before the wait.  volatile: it stays behind the wait in the program's order.
template <typename T>
__device__ __forceinline__ T mx_ld(const T* p) {
    T v;
    if constexpr (sizeof(T) == 16) {
        uint4& u = reinterpret_cast<uint4&>(v);
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    } else if constexpr (sizeof(T) == 4) {
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(reinterpret_cast<uint32_t&>(v)) : "l"(p));
    } else if constexpr (sizeof(T) == 1) {
        uint32_t byte;
        asm volatile("ld.global.u8 %0, [%1];" : "=r"(byte) : "l"(p));
        v = (T)byte;
    } else {
        static_assert(sizeof(T) == 2, "1, 2, 4 or 16 bytes");
        asm volatile("ld.global.b16 %0, [%1];" : "=h"(reinterpret_cast<uint16_t&>(v)) : "l"(p));
    }
    return v;
}

// What a lane of the encoders holds: 64 bytes as they were loaded, looked at only when they are
// needed.  That is a block of a 16-bit type, half a block of fp32 (the other half in the next lane).
template <typename T>
struct MxRaw {
    static constexpr int LANES = sizeof(T) / 2;            // lanes of a block
    static constexpr int N = 32 / LANES;                   // values of a lane
    uint32_t bits[16];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 16; ++i) bits[i] = 0u;
    }
    // `align`: of p, 32 or more, 16, or less.  Two 32-byte loads take each sector in one piece.
    __device__ __forceinline__ void load(const T* p, int align) {
        if (align >= 32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t* b = bits + 8 * h;
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7])
                             : "l"(p + 16 / LANES * h));
            }
        } else if (align >= 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = mx_ld(reinterpret_cast<const uint4*>(p) + i);
                bits[4 * i] = v.x, bits[4 * i + 1] = v.y, bits[4 * i + 2] = v.z, bits[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) reinterpret_cast<T*>(bits)[k] = mx_ld(p + k);
        }
    }
    // values 2i and 2i + 1
    __device__ __forceinline__ float2 pair(int i) const;
    // the largest magnitude, NaN if one is
    __device__ __forceinline__ float amax() const;
};

// the largest magnitude of three, NaN if one is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

template <>
__device__ __forceinline__ float2 MxRaw<float>::pair(int i) const {
    return make_float2(__uint_as_float(bits[2 * i]), __uint_as_float(bits[2 * i + 1]));
}
template <>
__device__ __forceinline__ float2 MxRaw<__half>::pair(int i) const {
    return __half22float2(*reinterpret_cast<const __half2*>(bits + i));
}
template <>
__device__ __forceinline__ float2 MxRaw<__nv_bfloat16>::pair(int i) const {
    return make_float2(__uint_as_float(bits[i] << 16), __uint_as_float(bits[i] & 0xffff0000u));
}
template <>
__device__ __forceinline__ float MxRaw<float>::amax() const {
    float m = __uint_as_float(bits[0]);
#pragma unroll
    for (int i = 1; i < 15; i += 2) m = max3_abs(m, __uint_as_float(bits[i]), __uint_as_float(bits[i + 1]));
    return max3_abs(m, __uint_as_float(bits[15]), __shfl_xor_sync(0xffffffffu, max3_abs(m, __uint_as_float(bits[15]), 0.0f), 1));
}
// two at a time; the signs of the running maximum mean nothing
template <>
__device__ __forceinline__ float MxRaw<__half>::amax() const {
    uint32_t m = bits[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(bits[i]));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max3_abs(v.x, v.y, 0.0f);
}
template <>
__device__ __forceinline__ float MxRaw<__nv_bfloat16>::amax() const {
    uint32_t m = bits[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(bits[i]));
    return max3_abs(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u), 0.0f);
}

// Encode a lane's values (the whole converged warp calls it): the codes in w, N / 2 bytes or, for
// E4M3, N; the block's scale byte returned.
template <bool E4M3, typename T>
__device__ __forceinline__ uint32_t mx_encode(const MxRaw<T>& raw, uint32_t (&w)[MxRaw<T>::N / (E4M3 ? 4 : 8)]) {
    constexpr int EMAX = E4M3 ? 8 : 2, N = MxRaw<T>::N;
    const int field = (int)(__float_as_uint(raw.amax()) >> 23);    // 255: the block holds an infinity or a NaN
    const int sf = max(field - EMAX, 0);                           // e + 127; 0 also where amax is 0 or subnormal
    // 2^-e = 2^(127 - sf): 127 - sf is -126 .. 127 for finite blocks
    const uint32_t inv = (uint32_t)(254 - sf) << 23;
    float2 t[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 v = raw.pair(i);
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
            "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "=f"(t[i].x), "=f"(t[i].y) : "f"(v.x), "f"(v.y), "f"(__uint_as_float(inv)));
    }
    if constexpr (E4M3) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h)
            asm("{\n\t.reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                "mov.b32 %0, {a, b};\n\t}"
                : "=r"(w[h]) : "f"(t[2 * h].x), "f"(t[2 * h].y), "f"(t[2 * h + 1].x), "f"(t[2 * h + 1].y));
    } else {
#pragma unroll
        for (int h = 0; h < N / 8; ++h)
            asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
                "mov.b32 %0, {a, b, c, d};\n\t}"
                : "=r"(w[h]) : "f"(t[4 * h].x), "f"(t[4 * h].y), "f"(t[4 * h + 1].x), "f"(t[4 * h + 1].y),
                  "f"(t[4 * h + 2].x), "f"(t[4 * h + 2].y), "f"(t[4 * h + 3].x), "f"(t[4 * h + 3].y));
    }
    if (field == 255)
#pragma unroll
        for (int h = 0; h < N / (E4M3 ? 4 : 8); ++h) w[h] = 0u;
    return field == 255 ? 255u : (uint32_t)sf;
}

// 8, 16 or 32 bytes in one store
template <int WORDS>
__device__ __forceinline__ void mx_put(uint8_t* p, const uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// n / d for 0 <= n < 2^31 and d >= 2 by a multiplication: with 2^(s - 1) < d <= 2^s and
// m = ceil(2^(31 + s) / d), which is below 2^32, n m / 2^(31 + s) is at least n / d and less than
// n / 2^(31 + s) <= 1 / d above it, too little to reach the next integer.
struct MxDivisor {
    uint32_t d, m, s;
};
inline MxDivisor mx_divisor(uint32_t d) {
    MxDivisor v{d, 0, 0};
    while ((1u << v.s) < d) ++v.s;
    v.m = (uint32_t)(((1ull << (31 + v.s)) + d - 1) / d);
    --v.s;                                                 // of the high half's shift
    return v;
}
__device__ __forceinline__ uint32_t mx_divide(uint32_t n, const MxDivisor& v) { return __umulhi(n, v.m) >> v.s; }

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
__device__ __forceinline__ void mx_segments(const int32_t* first, int n_experts, int64_t n_rows, int bn,
                                            int64_t max_groups, int* start, int* base, int* tmp) {
    const int per = (n_experts + (int)blockDim.x - 1) / (int)blockDim.x;
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, n_experts);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto at = [&](int e) { return (int)min(max((int64_t)mx_ld(first + e), (int64_t)0), n_rows); };
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
