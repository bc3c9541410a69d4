// Root-mean-square norm with the residual's addition and an 8-bit output (the layer's entry in
// front of a blockwise quantizer, HARP technical summary §2.4; codes and scales in codes.cuh):
//   h = rn_T(rn32(x + residual))              (h = x without a residual)
//   r = rn32(1 / sqrt(sum_j h_j^2 / d + eps)) (the sum, the quotient and the root in double)
//   u = rn32(rn32(h r) w)                     (w = 1 without a weight)
// and u's codes and scales, u itself rounded to T, or both.  One pass: a row stays in the
// registers of the threads that share it, between the sum and the codes.  The sum is taken
// in double so that r, and with it every code, does not depend on the order of addition (a sum of
// fp32 rounding errors would move r by an ulp from one launch shape to another); at 3 to 7 bytes per
// element in HBM its one conversion and one fused multiply-add stay hidden.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "codes.cuh"
#include "harp_internal.h"

namespace {

using namespace harp_codes;

struct NormParams {
    const void *x, *res, *w;
    int64_t rows, ld_x, ld_r;
    int d;
    double eps;
    void *h, *y;
    int64_t ld_h, ld_y;
    uint8_t* q;
    int64_t ld_q;
    float* s;
    int64_t ld_s;
    int qblock;
    bool vx, vr, vw, vh, vy, vq;   // vector access of each array
};

template <typename T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// blockDim.x threads share a row (a multiple of 32), blockDim.y rows per CTA; a thread holds N
// groups of 8 coordinates, group i at 8 (i blockDim.x + threadIdx.x).
template <typename T, typename C, int N>
__global__ void __launch_bounds__(1024) rms_norm_quant_kernel(const __grid_constant__ NormParams p) {
    __shared__ double part[32];
    const int tx = threadIdx.x, nx = blockDim.x;
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = r < p.rows;
    float v[N][8];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (i * nx + tx), n = live ? min(8, p.d - c) : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
        if (n > 0) load8((const T*)p.x + r * p.ld_x + c, n, p.vx, v[i]);
    }
    if (p.res) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (i * nx + tx), n = live ? min(8, p.d - c) : 0;
            if (n > 0) {
                float e[8];
                load8((const T*)p.res + r * p.ld_r + c, n, p.vr, e);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] = round_to<T>(v[i][k] + e[k]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (i * nx + tx), n = live ? min(8, p.d - c) : 0;
        if (p.h && n > 0) store8((T*)p.h + r * p.ld_h + c, n, p.vh, v[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double t = (double)v[i][k];
            sum = fma(t, t, sum);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (nx > 32) {
        const int wpr = nx >> 5, w0 = threadIdx.y * wpr;
        if ((tx & 31) == 0) part[w0 + (tx >> 5)] = sum;
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < wpr; ++w) sum += part[w0 + w];
    }
    const float rs = (float)(1.0 / sqrt(sum / (double)p.d + p.eps));
    const int qlanes = p.qblock / 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (i * nx + tx), n = live ? min(8, p.d - c) : 0;
        float a = 0.f;
        if (p.w) {
            float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (n > 0) load8((const T*)p.w + c, n, p.vw, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = __fmul_rn(__fmul_rn(v[i][k], rs), g[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = __fmul_rn(v[i][k], rs);
        }
        if (p.y && n > 0) store8((T*)p.y + r * p.ld_y + c, n, p.vy, v[i]);
        if (p.q) {
#pragma unroll
            for (int k = 0; k < 8; ++k) a = amax_nan(a, k < n ? v[i][k] : 0.f);
            for (int o = 1; o < qlanes; o <<= 1) a = amax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
            if (n > 0) {
                store_codes8<C>(p.q + r * p.ld_q + c, n, p.vq, v[i], code_factor<C>(a));
                if ((tx & (qlanes - 1)) == 0) p.s[r * p.ld_s + c / p.qblock] = code_scale<C>(a);
            }
        }
    }
}

template <typename T, typename C>
cudaError_t launch(const NormParams& p, int n, dim3 block, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.rows + block.y - 1) / block.y);
    switch (n) {
        case 1: rms_norm_quant_kernel<T, C, 1><<<grid, block, 0, stream>>>(p); break;
        case 2: rms_norm_quant_kernel<T, C, 2><<<grid, block, 0, stream>>>(p); break;
        default: rms_norm_quant_kernel<T, C, 4><<<grid, block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

bool aligned(const void* p, int64_t ld, size_t es, size_t to) {
    return (uintptr_t)p % to == 0 && ((size_t)ld * es) % to == 0;
}

}  // namespace

extern "C" harp_status harp_rms_norm_quant(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                                           const void* weight, int64_t rows, int64_t d, harp_dtype dtype, double eps,
                                           void* h, int64_t ld_h, void* y, int64_t ld_y, harp_code code, int32_t qblock,
                                           void* q, int64_t ld_q, float* scales, int64_t ld_s, void* stream) {
    harp_clear_error();
    if (dtype != HARP_F32 && dtype != HARP_BF16) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown dtype");
    if (code != HARP_CODE_I8 && code != HARP_CODE_E4M3) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown code format");
    if (rows < 0 || d < 1 || d > HARP_MAX_DIM) return harp_fail(HARP_ERR_INVALID_ARG, "rows >= 0 and 1 <= d <= 32768");
    if (rows > 0x7fffffffll) return harp_fail(HARP_ERR_INVALID_ARG, "more than 2^31 - 1 rows");
    // the lower end keeps 1 / sqrt(eps) finite in fp32, so that a zero row stays zero
    if (!(eps >= 1e-70) || eps > 1e30) return harp_fail(HARP_ERR_INVALID_ARG, "eps outside [1e-70, 1e30]");
    if (qblock != 32 && qblock != 64 && qblock != 128 && qblock != 256)
        return harp_fail(HARP_ERR_INVALID_ARG, "qblock must be 32, 64, 128 or 256");
    if (!q != !scales) return harp_fail(HARP_ERR_INVALID_ARG, "codes and scales go together");
    const int64_t nb = (d + qblock - 1) / qblock;
    if (ld_x < d || (residual && ld_r < d) || (h && ld_h < d) || (y && ld_y < d) || (q && (ld_q < d || ld_s < nb)))
        return harp_fail(HARP_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (rows == 0) return HARP_OK;
    if (!x || (!q && !y && !h)) return harp_fail(HARP_ERR_INVALID_ARG, "x is NULL or no output given");
    const size_t es = dtype == HARP_F32 ? 4 : 2;
    for (const void* v : {x, residual, weight, (const void*)h, (const void*)y})
        if ((uintptr_t)v % es) return harp_fail(HARP_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    if ((uintptr_t)scales % 4) return harp_fail(HARP_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    {
        // h may be x or the residual itself (a row is read whole before it is written); nothing
        // else that is written may share memory with anything
        struct Range {
            const void* p;
            size_t n;
            int64_t ld;
        };
        auto span = [&](int64_t ld, int64_t n, size_t e) { return ((size_t)(rows - 1) * ld + n) * e; };
        const Range in[3] = {{x, span(ld_x, d, es), ld_x}, {residual, span(ld_r, d, es), ld_r}, {weight, (size_t)d * es, -1}};
        const Range out[4] = {{h, span(ld_h, d, es), ld_h}, {y, span(ld_y, d, es), -1}, {q, span(ld_q, d, 1), -1},
                              {scales, span(ld_s, nb, 4), -1}};
        for (int o = 0; o < 4; ++o) {
            if (!out[o].p) continue;
            for (int i = 0; i < 3; ++i) {
                const bool in_place = o == 0 && i < 2 && out[o].p == in[i].p && out[o].ld == in[i].ld;
                if (in[i].p && !in_place && ranges_overlap(out[o].p, out[o].n, in[i].p, in[i].n))
                    return harp_fail(HARP_ERR_INVALID_ARG, "an output overlaps an input");
            }
            for (int k = 0; k < o; ++k)
                if (out[k].p && ranges_overlap(out[o].p, out[o].n, out[k].p, out[k].n))
                    return harp_fail(HARP_ERR_INVALID_ARG, "two outputs overlap");
        }
    }
    NormParams p;
    p.x = x, p.res = residual, p.w = weight;
    p.rows = rows, p.ld_x = ld_x, p.ld_r = ld_r;
    p.d = (int)d;
    p.eps = eps;
    p.h = h, p.y = y, p.ld_h = ld_h, p.ld_y = ld_y;
    p.q = (uint8_t*)q, p.ld_q = ld_q, p.s = scales, p.ld_s = ld_s;
    p.qblock = qblock;
    p.vx = aligned(x, ld_x, es, 16), p.vr = aligned(residual, ld_r, es, 16), p.vw = aligned(weight, 0, es, 16);
    p.vh = aligned(h, ld_h, es, 16), p.vy = aligned(y, ld_y, es, 16), p.vq = aligned(q, ld_q, 1, 8);
    // threads per row: as many as give each at most 4 groups of 8 coordinates; several short rows
    // share a CTA of 256 threads
    const int groups = (int)((d + 7) / 8);
    int nx = 32, n = 1;
    while (nx < 256 && nx < groups) nx *= 2;
    while (n < 4 && nx * n < groups) n *= 2;
    while (nx * n < groups) nx *= 2;
    const dim3 block((unsigned)nx, (unsigned)std::max(1, 256 / nx));
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == HARP_F32)
        e = code == HARP_CODE_I8 ? launch<float, CodeI8>(p, n, block, s) : launch<float, CodeE4M3>(p, n, block, s);
    else
        e = code == HARP_CODE_I8 ? launch<__nv_bfloat16, CodeI8>(p, n, block, s)
                                 : launch<__nv_bfloat16, CodeE4M3>(p, n, block, s);
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    harp_set_last_kernel("rms_norm_quant_kernel");
    return HARP_OK;
}
