// The 8-bit code formats of the blockwise quantizers: int8 (largest code 127) and e4m3
// (largest finite value 448), one fp32 scale per block.  For a block with maximum magnitude a:
//   s = a / Q, code = rne(v * (Q / a))          (each operation rounded to nearest in fp32)
// so v ~ code * s.  The product can exceed Q by one fp32 rounding, which both conversions
// round back to Q.  A block with a < 2^-100 counts as zero (s = 0, codes 0): Q / a stays finite
// and s normal.  A block that holds a NaN or an infinity keeps it in its scale, so every value
// it decodes to is NaN: nothing that was not finite comes back as a number.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace harp_codes {

constexpr float kZeroBlock = 7.888609052210118e-31f;   // 2^-100

// max of a and |v|; a NaN in either stays
__device__ __forceinline__ float amax_nan(float a, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(v)));
    return r;
}

// Four fp32 values as four codes in the bytes of a word, the first in the lowest byte.
struct CodeI8 {
    static constexpr float kTop = 127.f;
    static __device__ __forceinline__ uint32_t one(float v) {
        uint32_t r;
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(v));
        return r & 0xffu;
    }
    static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
        return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040), 0x5410);
    }
    static __device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = (float)(int)(int8_t)(w >> (8 * k));
    }
};

struct CodeE4M3 {
    static constexpr float kTop = 448.f;
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    static __device__ __forceinline__ uint32_t one(float v) { return two(v, 0.f) & 0xffu; }
    static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
        return two(a, b) | (two(c, d) << 16);
    }
    // e4m3 values are exact in fp16
    static __device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * k))));
            asm("{ .reg .f16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
                : "=f"(v[2 * k]), "=f"(v[2 * k + 1])
                : "r"(h));
        }
    }
};

// Q / a, the factor of a block's values (0 for a zero block, NaN and infinity)
template <typename C>
__device__ __forceinline__ float code_factor(float a) {
    return a >= kZeroBlock ? __fdiv_rn(C::kTop, a) : 0.f;
}
// a / Q, the block's scale (a NaN stays: the comparison is false for it)
template <typename C>
__device__ __forceinline__ float code_scale(float a) {
    return a < kZeroBlock ? 0.f : __fdiv_rn(a, C::kTop);
}

// Eight values of a row at p (elements e < n exist): 16-byte loads where `vec`, else one by one.
__device__ __forceinline__ void load8(const float* p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : 0.f;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? __bfloat162float(p[k]) : 0.f;
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store8(float* p, int n, bool vec, const float (&v)[8]) {
    if (vec && n >= 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = v[k];
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, bool vec, const float (&v)[8]) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = __float2bfloat16_rn(v[k]);
    }
}
// Eight codes: one 8-byte store where `vec`
template <typename C>
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, bool vec, const float (&v)[8], float factor) {
    const uint32_t lo = C::four(v[0] * factor, v[1] * factor, v[2] * factor, v[3] * factor);
    const uint32_t hi = C::four(v[4] * factor, v[5] * factor, v[6] * factor, v[7] * factor);
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = (uint8_t)((k < 4 ? lo : hi) >> (8 * (k & 3)));
    }
}

}  // namespace harp_codes
