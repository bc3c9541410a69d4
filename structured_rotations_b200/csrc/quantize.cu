// Blockwise 8-bit quantizer and its inverse (HARP technical summary §2.4: the rotation is a
// drop-in step in front of a blockwise quantizer; formats and arithmetic in codes.cuh).
//  * blocks of 1 x q, q = 32 .. 256: activation checkpoints for the calibration backward, and
//    the row operand of the e4m3 product;
//  * tiles of 128 x 128: the weight operand of the product.
// Both are one pass over the values in HBM: a thread keeps its values in registers between the
// block's maximum and the codes.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "codes.cuh"
#include "harp_internal.h"

namespace {

using namespace harp_codes;

constexpr int kThreads = 256;

struct QuantParams {
    const void* x;
    int64_t rows, cols, ld_x;
    uint8_t* q;
    int64_t ld_q;
    float* s;
    int64_t ld_s;
    int qblock, qshift;   // coordinates per block along a row, and their log2
    bool vx, vq;     // 16-byte loads of x, 8-byte stores of codes
};

// A warp's unit of work: N groups of 256 consecutive coordinates of a row.
struct Unit {
    int64_t r, c0;
};
template <int N>
__device__ __forceinline__ Unit unit_of(int64_t u, int64_t units, int64_t per_row) {
    int64_t r;
    if (units <= 0x7fffffff) r = (uint32_t)u / (uint32_t)per_row;
    else r = u / per_row;
    return {r, (u - r * per_row) * 256 * N};
}

// Blocks of 1 x q: 8 coordinates per lane, so a block is q / 8 lanes of a group.
template <typename T, typename C, int N>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
    const int64_t per_row = (p.cols + 256 * N - 1) / (256 * N), units = p.rows * per_row;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const Unit at = unit_of<N>(u, units, per_row);
        const T* x = (const T*)p.x + at.r * p.ld_x;
        Eight<T> x8[N];
        load_groups<T, N>(x, at.c0, 256, p.cols, p.vx, x8);
        quantize_groups<C, N>([&](int i, float(&v)[8]) { x8[i].get(v); }, at.c0, 256, p.cols, p.qblock / 8, p.q + at.r * p.ld_q, p.vq, p.s + at.r * p.ld_s);
    }
}

// Tiles of 128 x 128: a CTA per tile, 16 lanes across a row of the tile, 16 rows per pass.  HBM bounds it as long as
// enough tiles are under way: bf16 values stay packed, four CTAs per SM instead of two (28672 x 8192: 111
// us, 96 % of a copy, against 129, although 64 registers spill some 60 bytes; five CTAs spill more: 216).  fp32
// values take two CTAs' registers (28672 x 8192: 173 us, 6.8 TB/s).
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) quantize_tiles_kernel(const QuantParams p) {
    __shared__ float part[kThreads / 32];
    const int64_t tc = (p.cols + 127) / 128;
    const int64_t tr = (int64_t)blockIdx.x / tc, tj = (int64_t)blockIdx.x % tc;
    const int64_t c = tj * 128 + 8 * (threadIdx.x & 15), r0 = tr * 128 + (threadIdx.x >> 4);
    const int n = (int)max((int64_t)0, min((int64_t)8, p.cols - c));
    const bool whole = tj * 128 + 128 <= p.cols && tr * 128 + 128 <= p.rows;   // one path without conditions
    Eight<T> x[8];
    if (whole && p.vx) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i].load((const T*)p.x + (r0 + 16 * i) * p.ld_x + c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const int64_t r = r0 + 16 * i;
            if (n > 0 && r < p.rows) load8((const T*)p.x + r * p.ld_x + c, n, p.vx, v);
            x[i].set(v);   // values of T: exact
        }
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        x[i].get(v);
        a = amax_nan(a, amax8(v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = amax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a = amax_nan(a, part[w]);
    const float f = code_factor<C>(a);
    if (whole && p.vq) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            x[i].get(v);
            store_codes8<C>(p.q + (r0 + 16 * i) * p.ld_q + c, 8, true, v, f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 16 * i;
            float v[8];
            x[i].get(v);
            if (n > 0 && r < p.rows) store_codes8<C>(p.q + r * p.ld_q + c, n, p.vq, v, f);
        }
    }
    if (threadIdx.x == 0) p.s[tr * p.ld_s + tj] = code_scale<C>(a);
}

// y = rn(code * scale), 8 coordinates per lane (they share a block).
template <typename T, typename C, int N>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const QuantParams p, T* y, int brows) {
    const int lane = threadIdx.x & 31;
    const int64_t per_row = (p.cols + 256 * N - 1) / (256 * N), units = p.rows * per_row;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const Unit at = unit_of<N>(u, units, per_row);
        const uint8_t* q = p.q + at.r * p.ld_q;
        const float* sr = p.s + (brows == 1 ? at.r : at.r >> 7) * p.ld_s;
        uint32_t w[N][2];
        float s[N];
        Eight<T> y8[N];
        if (p.vq && whole_groups<N>(at.c0, 256, p.cols)) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t c = at.c0 + 256 * i + 8 * lane;
                const uint2 t = __ldcs(reinterpret_cast<const uint2*>(q + c));
                w[i][0] = t.x, w[i][1] = t.y;
                s[i] = __ldg(sr + (c >> p.qshift));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t c = at.c0 + 256 * i + 8 * lane;
                w[i][0] = w[i][1] = 0u, s[i] = 0.f;
                if (c < p.cols) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (c + k < p.cols) w[i][k >> 2] |= (uint32_t)q[c + k] << (8 * (k & 3));
                    s[i] = __ldg(sr + (c >> p.qshift));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a[4], b[4], v[8];
            C::decode4(w[i][0], a);
            C::decode4(w[i][1], b);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = a[k] * s[i], v[4 + k] = b[k] * s[i];
            if constexpr (sizeof(T) == 4 && !C::kNaN) {
                // the largest fp32 value's scale is rounded up: 127 of it is above that value again
                if (C::kTop * s[i] > 3.40282347e38f && s[i] <= 3.40282347e38f) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = copysignf(fminf(fabsf(v[k]), 3.40282347e38f), v[k]);
                }
            }
            y8[i].set(v);
        }
        store_groups<T, N>(y + at.r * p.ld_x, at.c0, 256, p.cols, p.vx, y8);
    }
}

harp_status check_block(int32_t brows, int32_t bcols) {
    if (brows == 1 && (bcols == 32 || bcols == 64 || bcols == 128 || bcols == 256)) return HARP_OK;
    if (brows == 128 && bcols == 128) return HARP_OK;
    return harp_fail(HARP_ERR_INVALID_ARG, "blocks are 1 x 32, 64, 128 or 256, or 128 x 128");
}

// The arguments that the two directions share: v is the matrix of values.
harp_status check_args(const void* v, int64_t rows, int64_t cols, int64_t ld, harp_dtype dtype, harp_code code,
                       int32_t brows, int32_t bcols, const void* q, int64_t ld_q, const void* s, int64_t ld_s) {
    if (dtype != HARP_F32 && dtype != HARP_BF16) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown dtype");
    if (code != HARP_CODE_I8 && code != HARP_CODE_E4M3) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown code format");
    if (rows < 0 || cols < 0) return harp_fail(HARP_ERR_INVALID_ARG, "rows or cols < 0");
    const harp_status st = check_block(brows, bcols);
    if (st != HARP_OK) return st;
    const int64_t sc = (cols + bcols - 1) / bcols, sr = (rows + brows - 1) / brows;
    if (ld < cols || ld_q < cols || ld_s < sc)
        return harp_fail(HARP_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (rows == 0 || cols == 0) return HARP_OK;
    if (!v || !q || !s) return harp_fail(HARP_ERR_INVALID_ARG, "a matrix, its codes or its scales are NULL");
    const size_t es = dtype == HARP_F32 ? 4 : 2;
    if ((uintptr_t)v % es || (uintptr_t)s % 4)
        return harp_fail(HARP_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    const size_t vb = ((size_t)(rows - 1) * ld + cols) * es, qb = (size_t)(rows - 1) * ld_q + cols,
                 sb = ((size_t)(sr - 1) * ld_s + sc) * sizeof(float);
    if (ranges_overlap(v, vb, q, qb) || ranges_overlap(v, vb, s, sb) || ranges_overlap(q, qb, s, sb))
        return harp_fail(HARP_ERR_INVALID_ARG, "values, codes and scales overlap");
    return HARP_OK;
}

QuantParams make_params(const void* v, int64_t rows, int64_t cols, int64_t ld, harp_dtype dtype, int32_t bcols,
                        const void* q, int64_t ld_q, const float* s, int64_t ld_s) {
    const size_t es = dtype == HARP_F32 ? 4 : 2;
    QuantParams p;
    p.x = v;
    p.rows = rows, p.cols = cols, p.ld_x = ld;
    p.q = (uint8_t*)const_cast<void*>(q);
    p.ld_q = ld_q;
    p.s = const_cast<float*>(s);
    p.ld_s = ld_s;
    p.qblock = bcols;
    p.qshift = bcols == 32 ? 5 : bcols == 64 ? 6 : bcols == 128 ? 7 : 8;
    // (a single row is never stepped past: its leading dimension plays no part)
    p.vx = (uintptr_t)v % 16 == 0 && (rows == 1 || (ld * es) % 16 == 0);
    p.vq = (uintptr_t)q % 8 == 0 && (rows == 1 || ld_q % 8 == 0);
    return p;
}

// Grid of warps that share `rows` rows in units of `width` coordinates.
unsigned unit_grid(int64_t rows, int64_t cols, int64_t width) {
    const int64_t units = rows * ((cols + width - 1) / width);
    return (unsigned)std::min<int64_t>((units + kThreads / 32 - 1) / (kThreads / 32), 32 * (int64_t)harp_sm_count());
}

// Units of four groups (1,024 coordinates: one lane's divisions serve 32 blocks of 32) where rows are long and
// there are enough units for every SM; else of one.
bool long_units(const QuantParams& p) {
    return p.cols > 512 && p.rows * ((p.cols + 1023) / 1024) >= 16 * (int64_t)harp_sm_count();
}

template <typename T, typename C>
harp_status run_quantize(const QuantParams& p, int32_t brows, cudaStream_t stream) {
    if (brows == 1) {
        if (long_units(p)) quantize_rows_kernel<T, C, 4><<<unit_grid(p.rows, p.cols, 1024), kThreads, 0, stream>>>(p);
        else quantize_rows_kernel<T, C, 1><<<unit_grid(p.rows, p.cols, 256), kThreads, 0, stream>>>(p);
    } else {
        const int64_t tiles = ((p.rows + 127) / 128) * ((p.cols + 127) / 128);
        if (tiles > 0x7fffffffll) return harp_fail(HARP_ERR_INVALID_ARG, "too many tiles");
        quantize_tiles_kernel<T, C><<<(unsigned)tiles, kThreads, 0, stream>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    harp_set_last_kernel(brows == 1 ? "quantize_rows_kernel" : "quantize_tiles_kernel");
    return HARP_OK;
}

template <typename T, typename C>
harp_status run_dequantize(const QuantParams& p, T* y, int32_t brows, cudaStream_t stream) {
    if (long_units(p)) dequantize_kernel<T, C, 4><<<unit_grid(p.rows, p.cols, 1024), kThreads, 0, stream>>>(p, y, brows);
    else dequantize_kernel<T, C, 1><<<unit_grid(p.rows, p.cols, 256), kThreads, 0, stream>>>(p, y, brows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    harp_set_last_kernel("dequantize_kernel");
    return HARP_OK;
}

}  // namespace

extern "C" harp_status harp_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, harp_dtype dtype,
                                     harp_code code, int32_t brows, int32_t bcols, void* q, int64_t ld_q, float* scales,
                                     int64_t ld_s, void* stream) {
    harp_clear_error();
    const harp_status st = check_args(x, rows, cols, ld_x, dtype, code, brows, bcols, q, ld_q, scales, ld_s);
    if (st != HARP_OK || rows == 0 || cols == 0) return st;
    const QuantParams p = make_params(x, rows, cols, ld_x, dtype, bcols, q, ld_q, scales, ld_s);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == HARP_F32)
        return code == HARP_CODE_I8 ? run_quantize<float, CodeI8>(p, brows, s) : run_quantize<float, CodeE4M3>(p, brows, s);
    return code == HARP_CODE_I8 ? run_quantize<__nv_bfloat16, CodeI8>(p, brows, s)
                                : run_quantize<__nv_bfloat16, CodeE4M3>(p, brows, s);
}

extern "C" harp_status harp_dequantize(const void* q, int64_t ld_q, const float* scales, int64_t ld_s, harp_code code,
                                       int32_t brows, int32_t bcols, int64_t rows, int64_t cols, void* y, int64_t ld_y,
                                       harp_dtype dtype, void* stream) {
    harp_clear_error();
    const harp_status st = check_args(y, rows, cols, ld_y, dtype, code, brows, bcols, q, ld_q, scales, ld_s);
    if (st != HARP_OK || rows == 0 || cols == 0) return st;
    const QuantParams p = make_params(y, rows, cols, ld_y, dtype, bcols, q, ld_q, scales, ld_s);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == HARP_F32)
        return code == HARP_CODE_I8 ? run_dequantize<float, CodeI8>(p, (float*)y, brows, s)
                                    : run_dequantize<float, CodeE4M3>(p, (float*)y, brows, s);
    return code == HARP_CODE_I8 ? run_dequantize<__nv_bfloat16, CodeI8>(p, (__nv_bfloat16*)y, brows, s)
                                : run_dequantize<__nv_bfloat16, CodeE4M3>(p, (__nv_bfloat16*)y, brows, s);
}
