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
// max |v| of eight values, a NaN kept; three operands per instruction
__device__ __forceinline__ float amax8(const float (&v)[8]) {
    auto max3 = [](float a, float b, float c) {
        float r;
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
        return r;
    };
    return max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7]));
}

// Two fp32 products by one instruction, each rounded to nearest.  (Sums stay single: a pair's sum behind a
// pair's product was made one fused operation, whose one rounding gave other int8 codes.)
__device__ __forceinline__ void mul2(float& x, float& y, float f) {
    asm("{ .reg .b64 a, b; mov.b64 a, {%0, %1}; mov.b64 b, {%2, %2}; mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "+f"(x), "+f"(y) : "f"(f));
}

// Four fp32 values as four codes in the bytes of a word, the first in the lowest byte.
struct CodeI8 {
    static constexpr float kTop = 127.f;
    static constexpr bool kNaN = false;
    // |v| <= 127 (1 + 2^-23): adding 1.5 2^23 rounds v to an integer, ties to even, in the low bits
    // (an addition where a conversion would take the slower pipe)
    static __device__ __forceinline__ uint32_t one(float v) { return __float_as_uint(__fadd_rn(v, 12582912.f)); }
    static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
        return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040), 0x5410);
    }
    // the byte, offset by 128, in the low bits of 2^23, less 2^23 + 128
    static __device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __fsub_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 + k)), 8388736.f);
    }
};

struct CodeE4M3 {
    static constexpr float kTop = 448.f;
    static constexpr bool kNaN = true;   // NaN keeps its code
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

// The same for values that every row reads (kept in the caches).
template <typename T>
__device__ __forceinline__ void load8_cached(const T* p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    } else {
        load8(p, n, false, v);
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
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = v[k];
#pragma unroll
    for (int k = 0; k < 8; k += 2) mul2(t[k], t[k + 1], factor);
    uint32_t lo = C::four(t[0], t[1], t[2], t[3]);
    uint32_t hi = C::four(t[4], t[5], t[6], t[7]);
    // int8 has no NaN: codes 0 in a block that is not finite (0 times its scale is NaN)
    if (!C::kNaN && factor == 0.f) lo = hi = 0u;
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = (uint8_t)((k < 4 ? lo : hi) >> (8 * (k & 3)));
    }
}

// N groups of 8 coordinates per lane of a warp: in group i the lanes hold the 256 consecutive coordinates
// from c0 + i step of a row of d (c0 and step multiples of 256).
//
// Whether all of them lie inside of the row: the whole warp then takes one path without conditions per
// lane, whose loads are issued together (conditional ones cost bf16 rows half of their speed).
template <int N>
__device__ __forceinline__ bool whole_groups(int64_t c0, int64_t step, int64_t d) {
    return c0 + (N - 1) * step + 256 <= d;
}

// Eight values as they lie in memory: half of the registers for bf16.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {   // rounded to nearest even
        a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
};

// The groups' values, zero behind the row's end.
template <typename T, int N>
__device__ __forceinline__ void load_groups(const T* row, int64_t c0, int64_t step, int64_t d, bool vec, Eight<T> (&x)[N]) {
    const int lane = threadIdx.x & 31;
    if (vec && whole_groups<N>(c0, step, d)) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i].load(row + c0 + i * step + 8 * lane);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = c0 + i * step + 8 * lane;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c < d) load8(row + c, (int)min((int64_t)8, d - c), vec, v);
            x[i].set(v);   // values of T: exact
        }
    }
}
template <typename T, int N>
__device__ __forceinline__ void store_groups(T* row, int64_t c0, int64_t step, int64_t d, bool vec, const Eight<T> (&x)[N]) {
    const int lane = threadIdx.x & 31;
    if (vec && whole_groups<N>(c0, step, d)) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i].store(row + c0 + i * step + 8 * lane);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = c0 + i * step + 8 * lane;
            float v[8];
            x[i].get(v);
            if (c < d) store8(row + c, (int)min((int64_t)8, d - c), vec, v);
        }
    }
}

// The groups' codes and scales.  get(i, v): group i's values, zero behind the row's end; it is asked twice, for
// the maximum and for the codes, so that the values need no registers in between.  A block is qlanes
// neighbouring lanes.  The two divisions of every block are made once, by one lane (lane L for the L-th of the warp's
// blocks), and handed round: per lane they would be most of the instructions.  q, s: the row's codes
// and scales.
template <typename C, int N, typename Get>
__device__ __forceinline__ void quantize_groups(const Get& get, int64_t c0, int64_t step, int64_t d, int qlanes,
                                                uint8_t* q, bool vec, float* s) {
    const int lane = threadIdx.x & 31, nb = 32 / qlanes;   // blocks of a group
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float v[8];
        get(i, v);
        a[i] = amax8(v);
    }
    for (int o = 1; o < qlanes; o <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = amax_nan(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
    }
    const int in = lane & (nb - 1), group = lane / nb;
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = __shfl_sync(0xffffffffu, a[i], in * qlanes);
        if (group == i) mine = t;
    }
    const float f = code_factor<C>(mine), sc = code_scale<C>(mine);
    {
        const int64_t c = c0 + group * step + 8 * in * qlanes;
        if (group < N && c < d) s[c / (8 * qlanes)] = sc;
    }
    float fi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) fi[i] = __shfl_sync(0xffffffffu, f, i * nb + lane / qlanes);
    if (vec && whole_groups<N>(c0, step, d)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            get(i, v);
            store_codes8<C>(q + c0 + i * step + 8 * lane, 8, true, v, fi[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = c0 + i * step + 8 * lane;
            float v[8];
            get(i, v);
            if (c < d) store_codes8<C>(q + c, (int)min((int64_t)8, d - c), vec, v, fi[i]);
        }
    }
}

}  // namespace harp_codes
