// The e4m3 product for many rows (prefill): persistent pairs of CTAs on 256 x NT tiles.
//
// Per block of 128 along k the pair multiplies 256 rows of x by NT rows of the weight with
// tcgen05.mma.cta_group::2 (each CTA holds its own 128 rows of x and half of the weight's tile, so
// every byte that it loads is used by both): 64 bytes of operands per SM and clock at the full
// e4m3 rate, against 96 for a CTA alone on 128 x 256.  The scales differ from block to
// block, so a block's sums cannot stay in tensor memory: they go into one of two buffers of NT
// columns, and while the tensor cores work on the next block, eight warps read the finished
// buffer, scale it and add it to fp32 sums in registers (128 per thread at NT = 256).
//   warps 0-7  sums: thread = one row of x (a lane of tensor memory) and NT / 2 columns
//   warp 8     TMA loads of this CTA's operands, completing on the leader's barrier
//   warp 9     tensor-memory allocation; in the leader (rank 0) tcgen05.mma for both CTAs
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "harp_internal.h"
#include "matmul.h"
#include "tc.cuh"

namespace {

using namespace harp_tc;

constexpr int kThreads = 384;
constexpr int kSumRegs = 232, kOtherRegs = 40;   // registers per thread after the split: 2 x 232 + 40 = 3 x 168 at launch
constexpr int kGroup = 16;   // tiles of rows that run together: their slices of x stay in L2 for every tile of the weight

template <int NT>
struct Shape {
    static constexpr int kA = 128 * 128, kB = NT / 2 * 128, kStageBytes = kA + kB;
    static constexpr int kStages = 6;
    static constexpr int kHalf = NT / 2;       // columns of a product: half of the tile
    static constexpr int kBuffers = 2;         // per half
    static constexpr int kCols = 2 * kBuffers * kHalf;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
};

struct TileOf {
    int64_t m, n;
};
// Tiles in groups of kGroup tiles of rows, rows fastest inside of a group.
__device__ __forceinline__ TileOf tile_of(int64_t t, int64_t mt, int64_t nt) {
    const int64_t per = kGroup * nt, g = t / per, in = t - g * per;
    const int64_t rows = min((int64_t)kGroup, mt - g * kGroup);
    return {g * kGroup + in % rows, in / rows};
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Row of N sums (c0 columns of n left): 32-byte stores where `vec`.
template <int N>
__device__ __forceinline__ void store_row(float* y, int64_t left, bool vec, const float (&v)[N]) {
    if (vec && left >= N) {
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[c + k]);
            store32(y + c, w);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < left) y[c] = v[c];
    }
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* y, int64_t left, bool vec, const float (&v)[N]) {
    if (vec && left >= N) {
#pragma unroll
        for (int c = 0; c < N; c += 16) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack2(v[c + 2 * k], v[c + 2 * k + 1]);
            store32(y + c, w);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < left) y[c] = __float2bfloat16_rn(v[c]);
    }
}

template <int NT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    matmul_tiles_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ MatmulParams p, int64_t mt, int64_t nt, bool vec, int* status) {
    using S = Shape<NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(stages + S::kStages * S::kStageBytes);
    uint64_t* empty = full + S::kStages;
    uint64_t* tfull = empty + S::kStages;
    uint64_t* tempty = tfull + 2 * S::kBuffers;   // both [half][buffer]
    uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2 * S::kBuffers);
    volatile int* failed = reinterpret_cast<volatile int*>(slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = mt * nt;
    const int kb = (int)p.kb;

    if (warp == 9) tmem_alloc<2>(slot, S::kCols);
    if (threadIdx.x == 256) {
        tma_prefetch(&map_x);
        tma_prefetch(&map_w);
        for (int i = 0; i < S::kStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
        for (int i = 0; i < 2 * S::kBuffers; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, 8);
        *failed = 0;
        mbar_init_fence();
    }
    fence_before();
    __syncthreads();
    cluster_sync();   // the barriers of both CTAs are ready
    fence_after();
    const uint32_t tmem = *slot;

    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == 8) {
        {
            int s = 0, ph = 0;
            int64_t used = 0;
            bool ok = true;
            for (int64_t t = pair; ok && t < tiles; t += pairs) {
                const TileOf at = tile_of(t, mt, nt);
                const int m0 = (int)(at.m * 256 + 128 * rank), n0 = (int)(at.n * NT + NT / 4 * rank);
                for (int k = 0; k < kb; ++k) {
                    if (used >= S::kStages && !(ok = mbar_wait_warp(empty + s, ph ^ 1, failed, status))) break;
                    unsigned char* st = stages + s * S::kStageBytes;
                    const uint32_t bar = map_to_rank(smem_u32(full + s), 0);
                    if (elect_one()) {
                    if (rank == 0) mbar_expect_tx(full + s, 2 * S::kStageBytes);
                    tma_load_pair(st, &map_x, k * 128, m0, bar);
                    tma_load_pair(st + S::kA, &map_w, k * 128, n0, bar);
                    tma_load_pair(st + S::kA + S::kB / 2, &map_w, k * 128, n0 + S::kHalf, bar);
                    }
                    __syncwarp();
                    ++used;
                    if (++s == S::kStages) s = 0, ph ^= 1;
                }
            }
            // the pair's last products have released every stage: no arrival on this CTA's barriers is left
            for (int i = 0; ok && i < S::kStages; ++i) {
                if (used >= S::kStages) ok = mbar_wait_warp(empty + s, ph ^ 1, failed, status);
                else if (i < used) ok = mbar_wait_warp(empty + i, 0, failed, status);
                if (++s == S::kStages) s = 0, ph ^= 1;
            }
        }
      } else if (warp == 9) {
        if (rank == 0) {
            int s = 0, ph = 0, b = 0, bph = 0;
            int64_t used = 0;
            bool ok = true;
            for (int64_t t = pair; ok && t < tiles; t += pairs) {
                for (int k = 0; k < kb; ++k) {
                    if (!(ok = mbar_wait_warp(full + s, ph, failed, status))) break;
                    const uint64_t a = operand_desc(stages + s * S::kStageBytes);
#pragma unroll
                    for (int h = 0; ok && h < 2; ++h) {
                        const int at = h * S::kBuffers + b;
                        if (used >= S::kBuffers && !(ok = mbar_wait_warp(tempty + at, bph ^ 1, failed, status))) break;
                        fence_after();
                        const uint64_t w = operand_desc(stages + s * S::kStageBytes + S::kA + h * S::kB / 2);
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma<2>(tmem + at * S::kHalf, a + 2 * i, w + 2 * i, instr_desc(256, S::kHalf), i > 0);
                            if (h == 1) mma_commit<2>(empty + s);
                            mma_commit<2>(tfull + at);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    ++used;
                    if (++s == S::kStages) s = 0, ph ^= 1;
                    if (++b == S::kBuffers) b = 0, bph ^= 1;
                }
            }
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        constexpr int N = NT / 2;   // columns of this thread
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        int b = 0, bph = 0;
        bool ok = true;
        for (int64_t t = pair; ok && t < tiles; t += pairs) {
            const TileOf at = tile_of(t, mt, nt);
            const int64_t r = at.m * 256 + 128 * rank + 32 * (warp & 3) + lane, c0 = at.n * NT + N * half;
            const bool row = r < p.rows;
            const float* sx = p.sx + (row ? r * p.ld_sx : 0);
            const float* sw = p.sw + min(c0, p.n - 1) / 128 * p.ld_sw;
            float sum[N];
#pragma unroll
            for (int c = 0; c < N; ++c) sum[c] = 0.f;
            // scales two blocks ahead of their use
            float x0 = row ? __ldg(sx) : 0.f, w0 = __ldg(sw), x1 = 0.f, w1 = 0.f;
            if (kb > 1) x1 = row ? __ldg(sx + 1) : 0.f, w1 = __ldg(sw + 1);
            for (int k = 0; k < kb; ++k) {
                float x2 = 0.f, w2 = 0.f;
                if (k + 2 < kb) x2 = row ? __ldg(sx + k + 2) : 0.f, w2 = __ldg(sw + k + 2);
                const int buf = half * S::kBuffers + b;
                ok = mbar_wait_warp(tfull + buf, bph, failed, status);
                if (!ok) break;
                fence_after();
                const float f = x0 * w0;
                x0 = x1, w0 = w1, x1 = x2, w1 = w2;
                const uint32_t addr = tmem + lanes + buf * S::kHalf;
                uint32_t u[32], v[32];
                tmem_ld(addr, u);
                tmem_ld(addr + 32, v);
                tmem_ld_wait(u);
                tmem_ld_wait(v);
#pragma unroll
                for (int c = 0; c < 32; c += 2) fma2(sum[c], sum[c + 1], u[c], u[c + 1], f);
                if constexpr (N == 128) {
                    tmem_ld(addr + 64, u);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) fma2(sum[32 + c], sum[33 + c], v[c], v[c + 1], f);
                    tmem_ld(addr + 96, v);
                    tmem_ld_wait(u);
                    tmem_ld_wait(v);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(tempty + buf), 0));
                if constexpr (N == 128) {
#pragma unroll
                    for (int c = 0; c < 32; c += 2) fma2(sum[64 + c], sum[65 + c], u[c], u[c + 1], f);
                }
#pragma unroll
                for (int c = 0; c < 32; c += 2) fma2(sum[N - 32 + c], sum[N - 31 + c], v[c], v[c + 1], f);
                if (++b == S::kBuffers) b = 0, bph ^= 1;
            }
            if (ok && row && c0 < p.n) store_row<N>((T*)p.y + r * p.ld_y + c0, p.n - c0, vec, sum);
        }
    }
    __syncwarp();
    __syncthreads();
    if (*failed) drain_delay();
    fence_before();
    cluster_sync();   // no arrival or product of the pair is under way
    fence_after();
    if (warp == 9) tmem_free<2>(tmem, S::kCols);
}

template <int NT, typename T>
harp_status launch(const MatmulParams& p, cudaStream_t stream) {
    using S = Shape<NT>;
    const int64_t mt = (p.rows + 255) / 256, nt = (p.n + NT - 1) / NT;
    CUtensorMap mx, mw;
    harp_status st;
    if ((st = matmul_tensor_map(&mx, p.x, p.rows, p.k, p.ld_x, 128)) != HARP_OK) return st;
    if ((st = matmul_tensor_map(&mw, p.w, p.n, p.k, p.ld_w, NT / 4)) != HARP_OK) return st;
    int* status = matmul_status_word();
    if (!status) return harp_fail(HARP_ERR_CUDA, "the device's status word has no address");
    const size_t es = sizeof(T);
    const bool vec = (uintptr_t)p.y % 32 == 0 && ((size_t)p.ld_y * es) % 32 == 0;
    auto kern = matmul_tiles_kernel<NT, T>;
    cudaError_t e = (cudaError_t)harp_set_smem_limit((const void*)kern, (int)S::kSmem);
    if (e == cudaSuccess) {
        const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(mt * nt, harp_sm_count() / 2));
        kern<<<(unsigned)(2 * pairs), kThreads, S::kSmem, stream>>>(mx, mw, p, mt, nt, vec, status);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    }
    harp_set_last_kernel("matmul_tiles_kernel");
    return HARP_OK;
}

}  // namespace

harp_status launch_matmul_tiles(const MatmulParams& p, harp_dtype out, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    return out == HARP_F32 ? launch<256, float>(p, s) : launch<256, __nv_bfloat16>(p, s);
}
