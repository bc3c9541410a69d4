// The e4m3 product for few rows (decode): tcgen05 with the weight as the M side of the tile.
//
// A CTA takes 128 rows of the weight (one tile of scales) and all rows of x, at most BT = 16 .. 128, so that the
// weight, whose bytes bound the call, is read once and no tensor-core tile is padded to 128 rows of
// x.  TMA brings 128-byte wide slices (one block of k) of both operands through a ring of stages;
// one thread issues the block's four products into one of several tensor-memory buffers; the
// other warps take the block's sums out of tensor memory, scale them with sx sw and add them up in
// fp32 registers while the next blocks' products run.  With few weight tiles a cluster of C CTAs
// splits k: each keeps the sums of its share, and they are added over distributed shared memory in
// the order of the ranks, so that equal calls give equal bits.
// Measured: 1 x 28672 x 8192 in 41 us, 5.7 TB/s of the weight's bytes (a copy: 6.5); 64 rows in 42; 24 x 5120 x
// 5120 in 9.7, where the launch, the first loads and the sum over the cluster count; all scales of a CTA
// loaded at its start instead of a block ahead: no faster.
//   warps 0-3  sums: thread = one weight row (a lane of tensor memory), BT registers
//   warp 4     TMA loads;  warp 5  tensor-memory allocation and tcgen05.mma
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "harp_internal.h"
#include "matmul.h"
#include "tc.cuh"

namespace {

using namespace harp_tc;

constexpr int kThreads = 192;

template <int BT>
struct Shape {
    static constexpr int kStageBytes = 128 * 128 + BT * 128;
    // two CTAs per SM up to BT = 64: 100 KB of stages each; one above
    static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 4 : 6;
    static constexpr int kBuffers = BT <= 64 ? 4 : 2;   // tensor-memory buffers of BT columns
    static constexpr int kCols = kBuffers * BT < 32 ? 32 : kBuffers * BT;
    static constexpr int kPerSm = BT <= 64 ? 2 : 1;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 4 * BT * 4 + 256;
};

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int BT, typename T>
__global__ void __launch_bounds__(kThreads, Shape<BT>::kPerSm)
    matmul_rows_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ MatmulParams p, int split, int* status,
                       const __grid_constant__ WaitLimit limit) {
    using S = Shape<BT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* ring = reinterpret_cast<float*>(stages + S::kStages * S::kStageBytes);   // [2][2][BT] factors
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + 4 * BT);
    uint64_t* empty = full + S::kStages;
    uint64_t* tfull = empty + S::kStages;
    uint64_t* tempty = tfull + S::kBuffers;
    uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + S::kBuffers);
    volatile int* failed = reinterpret_cast<volatile int*>(slot + 1);
    volatile int* odd = reinterpret_cast<volatile int*>(slot + 2);   // [2]: 1 + the last block whose scales are to be taken apart

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % split);
    const int64_t tile = blockIdx.x / split;
    const int64_t n0 = tile * 128;
    const int kb0 = (int)(p.kb * rank / split), kb1 = (int)(p.kb * (rank + 1) / split);

    if (warp == 5) tmem_alloc<1>(slot, S::kCols);
    if (threadIdx.x == 128) {
        tma_prefetch(&map_x);
        tma_prefetch(&map_w);
        for (int i = 0; i < S::kStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
        for (int i = 0; i < S::kBuffers; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, 4);
        *failed = odd[0] = odd[1] = 0;
        mbar_init_fence();
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *slot;
    // the prologue above ran beside the end of the stream's previous kernel, which may have made the
    // operands; everything below comes after it
    launch_dependents();
    wait_previous_grid();

    float sum[BT];
#pragma unroll
    for (int c = 0; c < BT; ++c) sum[c] = 0.f;

    if (warp == 4) {
        for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
            const int s = i % S::kStages;
            if (i >= S::kStages && !mbar_wait_warp(empty + s, ((i / S::kStages) & 1) ^ 1, failed, status, limit)) break;
            if (elect_one()) {
                unsigned char* st = stages + s * S::kStageBytes;
                mbar_expect_tx(full + s, S::kStageBytes + limit.extra_tx);
                tma_load(st, &map_w, kb * 128, (int)n0, full + s);
                tma_load(st + 128 * 128, &map_x, kb * 128, 0, full + s);
            }
            __syncwarp();
        }
    } else if (warp == 5) {
        for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
            const int s = i % S::kStages, b = i % S::kBuffers;
            if (!mbar_wait_warp(full + s, (i / S::kStages) & 1, failed, status, limit)) break;
            if (i >= S::kBuffers && !mbar_wait_warp(tempty + b, ((i / S::kBuffers) & 1) ^ 1, failed, status, limit)) break;
            fence_after();
            const uint64_t a = operand_desc(stages + s * S::kStageBytes);
            const uint64_t bd = operand_desc(stages + s * S::kStageBytes + 128 * 128);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma<1>(tmem + b * BT, a + 2 * k, bd + 2 * k, instr_desc(128, BT), k > 0);
                mma_commit<1>(empty + s);
                mma_commit<1>(tfull + b);
            }
            __syncwarp();
        }
    } else {
        // the factor of x's row `tid` for the next block: its scales loaded a block ahead, handed to the other
        // threads through the ring (where scales have to be taken apart, second, then first)
        const int tid = threadIdx.x;
        const bool has = tid < p.rows;
        const float* sx = p.sx + (has ? tid * p.ld_sx : 0);
        const float* sw = p.sw + tile * p.ld_sw;
        float next_x = 0.f, next_w = 0.f;
        if (has && kb0 < kb1) next_x = load_after_wait(sx + kb0), next_w = load_after_wait(sw + kb0);
        for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
            float* sc = ring + (i & 1) * 2 * BT;
            const float f = factor_or_nan(next_x, next_w);
            const int any = __any_sync(0xffffffffu, f != f);
            if (tid < BT) sc[tid] = f;
            if (any && lane == 0) odd[i & 1] = kb + 1;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const bool apart = odd[i & 1] == kb + 1;
            if (has && kb + 1 < kb1) next_x = load_after_wait(sx + kb + 1), next_w = load_after_wait(sw + kb + 1);
            if (apart) {   // hardly ever (all four warps agree, and meet again before any wait that may give up)
                const BlockFactor g = has ? block_factor(load_after_wait(sx + kb), load_after_wait(sw + kb)) : BlockFactor{1.f, 0.f};
                if (tid < BT) sc[tid] = g.second, sc[BT + tid] = g.first;
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            const int b = i % S::kBuffers;
            if (!mbar_wait_warp(tfull + b, (i / S::kBuffers) & 1, failed, status, limit)) {
                // it gave up: the warp goes on meeting the others at their barriers, no more
                for (int q = kb + 1; q < kb1; ++q) {
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (odd[(q - kb0) & 1] == q + 1) asm volatile("bar.sync 1, 128;" ::: "memory");
                }
                break;
            }
            fence_after();
            const uint32_t addr = tmem + ((uint32_t)(32 * warp) << 16) + b * BT;
            constexpr int W = BT < 32 ? 16 : 32;
            if (apart) {   // the sums meet one scale in tensor memory
#pragma unroll 1
                for (int c0 = 0; c0 < BT; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld(addr + c0, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * sc[BT + c0 + c]);
                    tmem_st(addr + c0, v);
                }
                tmem_st_wait();
            }
#pragma unroll
            for (int c0 = 0; c0 < BT; c0 += W) {
                uint32_t v[W];
                tmem_ld(addr + c0, v);
                tmem_ld_wait(v);
                if (c0 + W == BT) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty + b);
                }
#pragma unroll
                for (int c = 0; c < W; c += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sc + c0 + c);
                    sum[c0 + c] = fmaf(__uint_as_float(v[c]), f.x, sum[c0 + c]);
                    sum[c0 + c + 1] = fmaf(__uint_as_float(v[c + 1]), f.y, sum[c0 + c + 1]);
                    sum[c0 + c + 2] = fmaf(__uint_as_float(v[c + 2]), f.z, sum[c0 + c + 2]);
                    sum[c0 + c + 3] = fmaf(__uint_as_float(v[c + 3]), f.w, sum[c0 + c + 3]);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();   // every product has been read: the stages are free, no copy is in flight
    if (*failed) drain_delay();
    T* y = (T*)p.y;
    const int64_t j = n0 + threadIdx.x;
    if (split == 1) {
        if (warp < 4 && j < p.n) {
#pragma unroll
            for (int c = 0; c < BT; ++c)
                if (c < p.rows) put(y + c * p.ld_y + j, sum[c]);
        }
    } else {
        float* part = reinterpret_cast<float*>(stages);   // [BT][128]
        if (warp < 4) {
#pragma unroll
            for (int c = 0; c < BT; ++c) part[c * 128 + threadIdx.x] = sum[c];
        }
        cluster_sync();
        if (warp < 4) {
            for (int c = rank; c < BT; c += split) {
                if (c >= p.rows) break;
                const uint32_t at = smem_u32(part + c * 128 + threadIdx.x);
                float v = 0.f;
                for (int q = 0; q < split; ++q) {
                    float t;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(t) : "r"(map_to_rank(at, q)) : "memory");
                    v += t;
                }
                if (j < p.n) put(y + c * p.ld_y + j, v);
            }
        }
        cluster_sync();   // a CTA leaves when its partial sums have been read
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 5) tmem_free<1>(tmem, S::kCols);
}

template <int BT, typename T>
harp_status launch(const MatmulParams& p, cudaStream_t stream) {
    using S = Shape<BT>;
    const int64_t tiles = (p.n + 127) / 128;   // n < 2^31: at most 2^24, times at most 8
    // split k until the CTAs fill the SMs' slots (or a share would be under two blocks)
    const int64_t slots = (int64_t)S::kPerSm * harp_sm_count();
    int split = 1;
    while (split < 8 && tiles * split * 2 <= slots && p.kb >= 4 * split) split *= 2;
    CUtensorMap mx, mw;
    harp_status st;
    if ((st = matmul_tensor_map(&mx, p.x, p.rows, p.k, p.ld_x, BT)) != HARP_OK) return st;
    if ((st = matmul_tensor_map(&mw, p.w, p.n, p.k, p.ld_w, 128)) != HARP_OK) return st;
    int* status = matmul_status_word();
    if (!status) return harp_fail(HARP_ERR_CUDA, "the device's status word has no address");
    auto kern = matmul_rows_kernel<BT, T>;
    cudaError_t e = (cudaError_t)harp_set_smem_limit((const void*)kern, (int)S::kSmem);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tiles * split));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = S::kSmem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kern, mx, mw, p, split, status, matmul_wait_limit());
        if (e == cudaSuccess) e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    }
    harp_set_last_kernel("matmul_rows_kernel");
    return HARP_OK;
}

template <typename T>
harp_status launch_bt(const MatmulParams& p, cudaStream_t stream) {
    if (p.rows <= 16) return launch<16, T>(p, stream);
    if (p.rows <= 32) return launch<32, T>(p, stream);
    if (p.rows <= 64) return launch<64, T>(p, stream);
    return launch<128, T>(p, stream);
}

}  // namespace

harp_status launch_matmul_rows(const MatmulParams& p, harp_dtype out, void* stream) {
    return out == HARP_F32 ? launch_bt<float>(p, (cudaStream_t)stream) : launch_bt<__nv_bfloat16>(p, (cudaStream_t)stream);
}
