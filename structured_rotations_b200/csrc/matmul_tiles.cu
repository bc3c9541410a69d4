// The e4m3 product for many rows (prefill): persistent pairs of CTAs on 256 x NT tiles.
//
// Per block of 128 along k the pair multiplies 256 rows of x by NT rows of the weight with
// tcgen05.mma.cta_group::2 (each CTA holds its own 128 rows of x and half of the weight's tile, so
// every byte that it loads is used by both): at NT = 256, 64 bytes of operands per SM and clock at
// the full e4m3 rate, against 96 for a CTA alone on 128 x 256.  The scales differ from block to
// block, so a block's sums cannot stay in tensor memory: they go into one of 512 / NT buffers, and
// while the tensor cores work on the next blocks, eight warps read the finished buffer, scale it and
// add it to fp32 sums in registers (128 per thread at NT = 256).
//   warps 0-7  sums: thread = one row of x (a lane of tensor memory) and NT / 2 columns
//   warp 8     TMA loads of this CTA's operands, completing on the leader's barrier
//   warp 9     tensor-memory allocation; in the leader (rank 0) tcgen05.mma for both CTAs
//
// What bounds it, on 4096 x 28672 x 8192 (25 rounds of 64 blocks on 74 pairs): 0.90 ms in a burst (2.1 PFLOP/s; 1.05 under the
// power cap), 1.41 M clocks counted at 1.57 GHz, 884 a block, so either buffer is held for 1,768: for its
// products (512, the full rate), 270 until the waiting warps see them done, 370 until the leader sees the other
// CTA's arrivals, and some 610 for taking it into registers (half of the additions among the reads:
// registers do not hold a whole buffer beside the sums).  Copies of the kernel that leave out parts agree: 684 a
// block (0.75 ms) where the sums are read but not added, 617 (0.70 ms) where buffers go straight back, for
// which products and hand-over predict 576.  Ten warps are allocated as twelve, 168 registers each, and
// the 256-column kernel spills inside of the loop (80 bytes of loads with bf16 results, 4 with fp32 ones).
// Tried and no faster: halves of 128 columns with their own buffers, 192 columns with all loads before the
// additions, scales by another warp, results by TMA stores.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "harp_internal.h"
#include "matmul.h"
#include "tc.cuh"

namespace {

using namespace harp_tc;

constexpr int kThreads = 320;
constexpr int kGroup = 16;   // tiles of rows that run together: their slices of x stay in L2 for every tile of the weight

template <int NT>
struct Shape {
    static constexpr int kA = 128 * 128, kB = NT / 2 * 128, kStageBytes = kA + kB;
    static constexpr int kStages = NT == 256 ? 6 : 8;
    static constexpr int kBuffers = 512 / NT;
    static constexpr int kCols = kBuffers * NT;
    static constexpr int kOutFloats = 32 * 33;   // per warp: 32 rows x 32 results, padded
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 8 * kOutFloats * 4 + 256;
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
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 32 bytes of results, as one store where `wide` (32-byte aligned), else as two.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
template <int N>
__device__ __forceinline__ void store_row(float* y, const float (&v)[N], bool wide) {
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[c + k]);
        store32(y + c, w, wide);
    }
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* y, const float (&v)[N], bool wide) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack2(v[c + 2 * k], v[c + 2 * k + 1]);
        store32(y + c, w, wide);
    }
}

template <int NT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    matmul_tiles_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ MatmulParams p, int64_t mt, int64_t nt, int align_y, int* status,
                        const __grid_constant__ WaitLimit limit) {
    using S = Shape<NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* out = reinterpret_cast<float*>(stages + S::kStages * S::kStageBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(out + 8 * S::kOutFloats);
    uint64_t* empty = full + S::kStages;
    uint64_t* tfull = empty + S::kStages;
    uint64_t* tempty = tfull + S::kBuffers;
    uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + S::kBuffers);
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
        for (int i = 0; i < S::kBuffers; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, 16);
        *failed = 0;
        mbar_init_fence();
    }
    fence_before();
    __syncthreads();
    cluster_sync();   // the barriers of both CTAs are ready
    fence_after();
    const uint32_t tmem = *slot;

    if (warp == 8) {
        int s = 0, ph = 0;
        int64_t used = 0;
        bool ok = true;
        for (int64_t t = pair; ok && t < tiles; t += pairs) {
            const TileOf at = tile_of(t, mt, nt);
            const int m0 = (int)(at.m * 256 + 128 * rank), n0 = (int)(at.n * NT + NT / 2 * rank);
            for (int k = 0; k < kb; ++k) {
                if (used >= S::kStages && !(ok = mbar_wait_warp(empty + s, ph ^ 1, failed, status, limit))) break;
                if (elect_one()) {
                    unsigned char* st = stages + s * S::kStageBytes;
                    const uint32_t bar = map_to_rank(smem_u32(full + s), 0);
                    if (rank == 0) mbar_expect_tx(full + s, 2 * S::kStageBytes + limit.extra_tx);
                    tma_load_pair(st, &map_x, k * 128, m0, bar);
                    tma_load_pair(st + S::kA, &map_w, k * 128, n0, bar);
                }
                __syncwarp();
                ++used;
                if (++s == S::kStages) s = 0, ph ^= 1;
            }
        }
        // the pair's last products have released every stage: no arrival on this CTA's barriers is left
        for (int i = 0; ok && i < S::kStages; ++i) {
            if (used >= S::kStages) ok = mbar_wait_warp(empty + s, ph ^ 1, failed, status, limit);
            else if (i < used) ok = mbar_wait_warp(empty + i, 0, failed, status, limit);
            if (++s == S::kStages) s = 0, ph ^= 1;
        }
    } else if (warp == 9) {
        int s = 0, ph = 0, b = 0, bph = 0;
        int64_t used = 0;
        bool ok = true, ready = false;   // ready: the next stage was seen full while the last products were issued
        for (int64_t t = pair; ok && rank == 0 && t < tiles; t += pairs) {
            for (int k = 0; k < kb; ++k) {
                if (!ready && !(ok = mbar_wait_warp(full + s, ph, failed, status, limit))) break;
                if (used >= S::kBuffers && !(ok = mbar_wait_warp(tempty + b, bph ^ 1, failed, status, limit))) break;
                fence_after();
                if (elect_one()) {
                    const uint64_t a = operand_desc(stages + s * S::kStageBytes);
                    const uint64_t w = operand_desc(stages + s * S::kStageBytes + S::kA);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma<2>(tmem + b * NT, a + 2 * i, w + 2 * i, instr_desc(256, NT), i > 0);
                    mma_commit<2>(tfull + b);
                    mma_commit<2>(empty + s);
                }
                __syncwarp();
                ++used;
                if (++s == S::kStages) s = 0, ph ^= 1;
                if (++b == S::kBuffers) b = 0, bph ^= 1;
                ready = mbar_test_warp(full + s, ph);
            }
        }
    } else {
        constexpr int N = NT / 2;   // columns of this thread
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        float* mine = out + warp * S::kOutFloats;
        const uint32_t back = map_to_rank(smem_u32(tempty), 0);
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
            // scales a block ahead of their use
            float x1 = row ? __ldg(sx) : 0.f, w1 = __ldg(sw);
            for (int k = 0; k < kb; ++k) {
                float f = factor_or_nan(x1, w1);
                const bool apart = __any_sync(0xffffffffu, f != f);
                if (k + 1 < kb) x1 = row ? __ldg(sx + k + 1) : 0.f, w1 = __ldg(sw + k + 1);
                ok = mbar_wait_warp(tfull + b, bph, failed, status, limit);
                if (!ok) break;
                fence_after();
                const uint32_t addr = tmem + lanes + b * NT + N * half;
                uint32_t v[2][16];
                if (apart) {   // hardly ever: the sums meet one scale in tensor memory
                    const BlockFactor g = block_factor(row ? __ldg(sx + k) : 0.f, __ldg(sw + k));
#pragma unroll 1
                    for (int c = 0; c < N; c += 16) {
                        tmem_ld(addr + c, v[0]);
                        tmem_ld_wait(v[0]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[0][j] = __float_as_uint(__uint_as_float(v[0][j]) * g.first);
                        tmem_st(addr + c, v[0]);
                    }
                    tmem_st_wait();
                    f = g.second;
                }
                tmem_ld(addr, v[0]);
#pragma unroll
                for (int i = 0; i < N / 16; ++i) {
                    tmem_ld_wait(v[i & 1]);
                    if (i + 1 < N / 16) {
                        tmem_ld(addr + 16 * (i + 1), v[(i + 1) & 1]);
                    } else {
                        fence_before();
                        __syncwarp();
                        if (elect_one()) mbar_arrive_cluster(back + 8 * b);
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) fma2(sum[16 * i + c], sum[16 * i + c + 1], v[i & 1][c], v[i & 1][c + 1], f);
                }
                if (++b == S::kBuffers) b = 0, bph ^= 1;
            }
            if (!ok) break;
            if (c0 >= p.n) continue;
            if (align_y >= 16 && c0 + N <= p.n) {
                if (row) store_row((T*)p.y + r * p.ld_y + c0, sum, align_y >= 32);
                continue;
            }
            // 32 columns at a time through shared memory: a row's 32 consecutive results per store (4000 x 28001 x
            // 4096: 476 us; two rows of 16 each: 555)
            const int64_t r0 = r - lane;
            const int live = (int)max((int64_t)0, min((int64_t)32, p.rows - r0));
#pragma unroll
            for (int i = 0; i < N / 32; ++i) {
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 32; ++c) mine[lane * 33 + c] = sum[32 * i + c];
                __syncwarp();
                const int64_t c = c0 + 32 * i + lane;
                if (c < p.n) {
                    T* y = (T*)p.y + r0 * p.ld_y + c;
#pragma unroll 8
                    for (int j = 0; j < live; ++j, y += p.ld_y) put(y, mine[j * 33 + lane]);
                }
            }
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
    if ((st = matmul_tensor_map(&mw, p.w, p.n, p.k, p.ld_w, NT / 2)) != HARP_OK) return st;
    int* status = matmul_status_word();
    if (!status) return harp_fail(HARP_ERR_CUDA, "the device's status word has no address");
    const uint64_t to = (uint64_t)(uintptr_t)p.y | (uint64_t)p.ld_y * sizeof(T);
    const int align_y = to % 32 == 0 ? 32 : to % 16 == 0 ? 16 : 1;
    auto kern = matmul_tiles_kernel<NT, T>;
    cudaError_t e = (cudaError_t)harp_set_smem_limit((const void*)kern, (int)S::kSmem);
    if (e == cudaSuccess) {
        const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(mt * nt, harp_sm_count() / 2));
        kern<<<(unsigned)(2 * pairs), kThreads, S::kSmem, stream>>>(mx, mw, p, mt, nt, align_y, status, matmul_wait_limit());
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
    // The narrower tile where it leaves fewer pairs idle: a block of 256 x 128 takes about 0.6 of the time of
    // one of 256 x 256, so with t tiles of 256 columns on P pairs it wins when ceil(2 t / P) 0.6 < ceil(t / P).
    const int64_t pairs = std::max(1, harp_sm_count() / 2), mt = (p.rows + 255) / 256;
    const int64_t wide = (mt * ((p.n + 255) / 256) + pairs - 1) / pairs, narrow = (mt * ((p.n + 127) / 128) + pairs - 1) / pairs;
    if (3 * narrow < 5 * wide)
        return out == HARP_F32 ? launch<128, float>(p, s) : launch<128, __nv_bfloat16>(p, s);
    return out == HARP_F32 ? launch<256, float>(p, s) : launch<256, __nv_bfloat16>(p, s);
}
