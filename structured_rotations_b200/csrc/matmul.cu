// Matrix product of e4m3 codes with fp32 scales per block of 128 (the rotated rows times the
// rotated weight, both quantized: HARP technical summary §2.4):
//   y[r][j] = sum_kb sx[r][kb] sw[j / 128][kb] sum_{i in block kb} x[r][i] w[j][i]
// matmul_simple_kernel takes any alignment: a CTA computes 64 x 64 results, the codes of a
// 32-wide slice of k decoded to fp32 in shared memory, each thread 4 x 4 fp32 sums per block of
// 128, which are scaled and added up in fp32 at the block's end.
// matmul_rows.cu holds the tensor-core kernel for few rows, matmul_tiles.cu the one for many.
#include <algorithm>
#include <atomic>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "codes.cuh"
#include "harp_internal.h"
#include "matmul.h"

namespace {

constexpr int kThreads = 256, kTile = 64, kSlice = 32;

__device__ __forceinline__ float decode(uint8_t c) {
    float v[4];
    harp_codes::CodeE4M3::decode4(c, v);
    return v[0];
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) matmul_simple_kernel(const MatmulParams p) {
    __shared__ float xs[kSlice][kTile + 4], ws[kSlice][kTile + 4];
    const int64_t j0 = (int64_t)blockIdx.x * kTile, r0 = (int64_t)blockIdx.y * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float y[4][4] = {};
    for (int64_t kb = 0; kb < p.kb; ++kb) {
        float t[4][4] = {};
        const int64_t kend = min(p.k, (kb + 1) * 128);
        for (int64_t k0 = kb * 128; k0 < kend; k0 += kSlice) {
            for (int e = threadIdx.x; e < kTile * kSlice; e += kThreads) {
                const int k = e % kSlice, i = e / kSlice;
                const bool in = k0 + k < kend;
                xs[k][i] = in && r0 + i < p.rows ? decode(p.x[(r0 + i) * p.ld_x + k0 + k]) : 0.f;
                ws[k][i] = in && j0 + i < p.n ? decode(p.w[(j0 + i) * p.ld_w + k0 + k]) : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kSlice; ++k) {
                float a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = xs[k][4 * ty + i], b[i] = ws[k][4 * tx + i];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = fmaf(a[i], b[j], t[i][j]);
            }
            __syncthreads();
        }
        const float sw = p.sw[(j0 / 128) * p.ld_sw + kb];   // 64 results of a tile lie in one block of 128
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 4 * ty + i;
            const BlockFactor s = block_factor(r < p.rows ? p.sx[r * p.ld_sx + kb] : 0.f, sw);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = fmaf(t[i][j] * s.first, s.second, y[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 4 * ty + i, c = j0 + 4 * tx + j;
            if (r < p.rows && c < p.n) put((T*)p.y + r * p.ld_y + c, y[i][j]);
        }
}

harp_status launch_simple(const MatmulParams& p, harp_dtype out, cudaStream_t stream) {
    const int64_t gx = (p.n + kTile - 1) / kTile;
    if (gx > 0x7fffffffll) return harp_fail(HARP_ERR_INVALID_ARG, "n too large");
    // the grid's second dimension holds 65,535 tiles of rows: longer batches in several launches
    const int64_t step = 65535ll * kTile;
    for (int64_t r = 0; r < p.rows; r += step) {
        MatmulParams q = p;
        const size_t es = out == HARP_F32 ? 4 : 2;
        q.x += r * p.ld_x, q.sx += r * p.ld_sx, q.y = (char*)p.y + (size_t)r * p.ld_y * es;
        q.rows = std::min(step, p.rows - r);
        const dim3 grid((unsigned)gx, (unsigned)((q.rows + kTile - 1) / kTile));
        if (out == HARP_F32) matmul_simple_kernel<float><<<grid, kThreads, 0, stream>>>(q);
        else matmul_simple_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    }
    harp_set_last_kernel("matmul_simple_kernel");
    return HARP_OK;
}

// set by a bounded wait that gave up (harp_device_status)
__device__ int g_wait_status;

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &res) == cudaSuccess &&
            res == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        cudaGetLastError();
    });
    return fn;
}

}  // namespace

harp_status matmul_tensor_map(CUtensorMap* map, const void* q, int64_t rows, int64_t k, int64_t ld, int box_rows) {
    auto encode = encoder();
    if (!encode) return harp_fail(HARP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dim[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t stride[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1, 1};
    auto run = [&] {
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dim, stride, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = run();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // a host thread whose first CUDA call this is has no current context yet
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) cudaGetLastError();
        r = run();
    }
    if (r != CUDA_SUCCESS) return harp_fail(HARP_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
    return HARP_OK;
}

int* matmul_status_word() {
    static std::atomic<int*> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return nullptr;
    }
    int* p = cached[dev].load(std::memory_order_relaxed);
    if (!p) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_wait_status) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        p = (int*)a;
        cached[dev].store(p, std::memory_order_relaxed);
    }
    return p;
}

harp_tc::WaitLimit matmul_wait_limit() {
    const WaitInjection w = harp_wait_injection();
    return {w.extra_bytes ? (long long)w.limit : harp_tc::kWaitClocks, w.extra_bytes};
}

extern "C" harp_status harp_device_status(void) {
    harp_clear_error();
    int* word = matmul_status_word();
    if (!word) return harp_fail(HARP_ERR_CUDA, "no CUDA device");
    int v = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&v, word, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) e = cudaMemset(word, 0, sizeof v);
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    return v ? harp_fail(HARP_ERR_TIMEOUT, "a bounded device-side wait gave up") : HARP_OK;
}

extern "C" harp_status harp_matmul_quant(const void* x, int64_t ld_x, const float* sx, int64_t ld_sx, const void* w,
                                         int64_t ld_w, const float* sw, int64_t ld_sw, int64_t rows, int64_t n,
                                         int64_t k, void* y, int64_t ld_y, harp_dtype out_dtype, void* stream) {
    harp_clear_error();
    if (out_dtype != HARP_F32 && out_dtype != HARP_BF16) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown dtype");
    if (rows < 0 || n < 0 || k < 1) return harp_fail(HARP_ERR_INVALID_ARG, "rows >= 0, n >= 0 and k >= 1");
    if (rows > 0x7fffffffll || n > 0x7fffffffll || k > 0x7fffffffll)
        return harp_fail(HARP_ERR_INVALID_ARG, "a side of the product above 2^31 - 1");
    const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128;
    if (ld_x < k || ld_w < k || ld_sx < kb || ld_sw < kb || ld_y < n)
        return harp_fail(HARP_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if (rows == 0 || n == 0) return HARP_OK;
    if (!x || !sx || !w || !sw || !y) return harp_fail(HARP_ERR_INVALID_ARG, "an operand or the result is NULL");
    const size_t es = out_dtype == HARP_F32 ? 4 : 2;
    if ((uintptr_t)sx % 4 || (uintptr_t)sw % 4 || (uintptr_t)y % es)
        return harp_fail(HARP_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    const size_t yb = ((size_t)(rows - 1) * ld_y + n) * es;
    if (ranges_overlap(y, yb, x, (size_t)(rows - 1) * ld_x + k) || ranges_overlap(y, yb, w, (size_t)(n - 1) * ld_w + k) ||
        ranges_overlap(y, yb, sx, ((size_t)(rows - 1) * ld_sx + kb) * 4) ||
        ranges_overlap(y, yb, sw, ((size_t)(nb - 1) * ld_sw + kb) * 4))
        return harp_fail(HARP_ERR_INVALID_ARG, "the result overlaps an operand");
    // a single row is never stepped past: its leading dimension plays no part in the alignment
    const int64_t whole = (k + 15) / 16 * 16;
    if (rows == 1) ld_x = whole;
    if (n == 1) ld_w = whole;
    const MatmulParams p{(const uint8_t*)x, (const uint8_t*)w, sx, sw, y, ld_x, ld_w, ld_sx, ld_sw, ld_y, rows, n, k, kb};
    // TMA takes 16-byte aligned operands whose rows are a multiple of 16 bytes (below 2^40) apart
    const bool tma = ((uintptr_t)x | (uintptr_t)w | (uintptr_t)ld_x | (uintptr_t)ld_w) % 16 == 0 && ld_x < (1ll << 40) &&
                     ld_w < (1ll << 40);
    if (tma) {
        // Up to 64 rows the weight's bytes count and the rows kernel streams them with every SM (64 x 28672 x
        // 8192: 45 us against 67); from there the pair kernel multiplies faster (128 x 4096 x 4096: 14.7 us
        // against 18.5), unless up to 128 rows meet so few columns that most pairs would idle while
        // the rows kernel splits k (128 x 1024 x 8192: 13.4 us against 24.5).
        const bool few = rows <= 64 || (rows <= 128 && (n + 127) / 128 <= harp_sm_count() / 8);
        return few ? launch_matmul_rows(p, out_dtype, stream) : launch_matmul_tiles(p, out_dtype, stream);
    }
    return launch_simple(p, out_dtype, (cudaStream_t)stream);
}
