// Root-mean-square norm with the residual's addition and an 8-bit output (the layer's entry in
// front of a blockwise quantizer, HARP technical summary §2.4; codes and scales in codes.cuh):
//   h = rn_T(rn32(x + residual))              (h = x without a residual)
//   r = rn32(1 / sqrt(sum_j h_j^2 / d + eps)) (the sum, its mean and the root in double)
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
    double eps, inv_d;
    void *h, *y;
    int64_t ld_h, ld_y;
    uint8_t* q;
    int64_t ld_q;
    float* s;
    int64_t ld_s;
    int qblock;
    bool vx, vr, vw, vh, vy, vq;   // vector access of each array
};

// blockDim.x threads share a row (a multiple of 32), blockDim.y rows per CTA of at most MOST threads; a thread holds N
// groups of 8 coordinates, group i at 8 (i blockDim.x + threadIdx.x).
template <typename T, typename C, int N, int MOST>
__global__ void __launch_bounds__(MOST) rms_norm_quant_kernel(const __grid_constant__ NormParams p) {
    __shared__ double part[32];
    const int tx = threadIdx.x, nx = blockDim.x;
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = r < p.rows;
    const int64_t c0 = 8 * (tx & ~31), step = 8 * nx;
    Eight<T> h8[N];   // the row's sum, in T
    double sum = 0.0;
    if (live) {
        load_groups<T, N>((const T*)p.x + r * p.ld_x, c0, step, p.d, p.vx, h8);
        if (p.res) {
            Eight<T> e8[N];
            load_groups<T, N>((const T*)p.res + r * p.ld_r, c0, step, p.d, p.vr, e8);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[8], e[8];
                h8[i].get(v);
                e8[i].get(e);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += e[k];
                h8[i].set(v);
            }
        }
        if (p.h) store_groups<T, N>((T*)p.h + r * p.ld_h, c0, step, p.d, p.vh, h8);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            h8[i].get(v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const double t = (double)v[k];
                sum = fma(t, t, sum);
            }
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
    const float rs = (float)rsqrt(sum * p.inv_d + p.eps);
    if (!live) return;
    // group i of u
    const bool whole = whole_groups<N>(c0, step, p.d);
    auto u = [&](int i, float(&v)[8]) {
        h8[i].get(v);
        const int c = 8 * (i * nx + tx);
        if (p.w) {
            float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (whole || c < p.d) load8_cached((const T*)p.w + c, whole ? 8 : min(8, p.d - c), p.vw, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(__fmul_rn(v[k], rs), g[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], rs);
        }
        if (!whole) {   // nothing there takes part in the row's last block, a NaN row's zeros neither
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k >= p.d) v[k] = 0.f;
        }
    };
    float v[N][8];   // kept: computing u again for the codes took 0.24 ms instead of 0.21 (with a weight, d = 5120)
#pragma unroll
    for (int i = 0; i < N; ++i) u(i, v[i]);
    auto kept = [&](int i, float(&o)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = v[i][k];
    };
    if (p.y) {
        Eight<T> y8[N];
#pragma unroll
        for (int i = 0; i < N; ++i) y8[i].set(v[i]);
        store_groups<T, N>((T*)p.y + r * p.ld_y, c0, step, p.d, p.vy, y8);
    }
    if (p.q) quantize_groups<C, N>(kept, c0, step, p.d, p.qblock / 8, p.q + r * p.ld_q, p.vq, p.s + r * p.ld_s);
}

template <typename T, typename C>
cudaError_t launch(const NormParams& p, int n, dim3 block, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.rows + block.y - 1) / block.y);
    if (n == 1) rms_norm_quant_kernel<T, C, 1, 1024><<<grid, block, 0, stream>>>(p);
    else if (n == 2) rms_norm_quant_kernel<T, C, 2, 256><<<grid, block, 0, stream>>>(p);
    else if (block.x * block.y <= 256) rms_norm_quant_kernel<T, C, 4, 256><<<grid, block, 0, stream>>>(p);
    else rms_norm_quant_kernel<T, C, 4, 1024><<<grid, block, 0, stream>>>(p);
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
                const bool in_place = o == 0 && i < 2 && out[o].p == in[i].p && (rows == 1 || out[o].ld == in[i].ld);
                if (in[i].p && !in_place && ranges_overlap(out[o].p, out[o].n, in[i].p, in[i].n))
                    return harp_fail(HARP_ERR_INVALID_ARG, "an output overlaps an input");
            }
            for (int k = 0; k < o; ++k)
                if (out[k].p && ranges_overlap(out[o].p, out[o].n, out[k].p, out[k].n))
                    return harp_fail(HARP_ERR_INVALID_ARG, "two outputs overlap");
        }
    }
    if (rows == 1) ld_x = ld_r = ld_h = ld_y = ld_q = 0;   // a single row is never stepped past: any alignment of its end will do
    NormParams p;
    p.x = x, p.res = residual, p.w = weight;
    p.rows = rows, p.ld_x = ld_x, p.ld_r = ld_r;
    p.d = (int)d;
    p.eps = eps, p.inv_d = 1.0 / (double)d;
    p.h = h, p.y = y, p.ld_h = ld_h, p.ld_y = ld_y;
    p.q = (uint8_t*)q, p.ld_q = ld_q, p.s = scales, p.ld_s = ld_s;
    p.qblock = qblock;
    p.vx = aligned(x, ld_x, es, 16), p.vr = aligned(residual, ld_r, es, 16), p.vw = aligned(weight, 0, es, 16);
    p.vh = aligned(h, ld_h, es, 16), p.vy = aligned(y, ld_y, es, 16), p.vq = aligned(q, ld_q, 1, 8);
    // Four groups of 8 coordinates per thread, which keeps enough loads of enough rows under way; one where
    // the rows leave SMs idle; several short rows to a CTA of 256 threads.
    const int groups = (int)((d + 7) / 8);
    // (fp32 rows above 8,192 coordinates take more than 256 threads at 64 registers and spill 164 bytes: 8192 x 16384 with
    // residual 283 us, 6.2 TB/s.)
    const int n = rows <= harp_sm_count() && groups <= 1024 ? 1 : groups <= 64 ? 2 : 4;
    const int nx = (groups + 32 * n - 1) / (32 * n) * 32;
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
