// Calibration backward of the HARP transform (HARP technical summary §2.3 Optimization
// Objective: the parameters are fitted per layer from calibration data, which needs the
// gradient of the fit's loss through the transform).  For rows x_r and upstream gradients
// g_r = dL/dy_r of y_r = T x_r, harp_grad_theta returns dL/dtheta.
//
// Two kernels:
//  1. harp_grad_blocks_kernel: dL/dB_{t,c} = sum_r h_{t+1,r}[group] z_{t,r}[group]^T, with
//     z_t the input of stage t and h_{t+1} the gradient at its output.  A persistent CTA
//     takes tiles of R rows; per tile it holds x and g in shared memory as fp32, runs the
//     stages but the last forward on x, then walks them backwards: in one pass over each
//     group it recovers the stage's input through the transposed block (z_t = B^T z_{t+1},
//     exact up to rounding because B is orthogonal, so no intermediate is stored; the last
//     stage's input is still there), adds the outer products h (x) z over the tile's rows, and
//     moves the gradient down (h_t = B^T h_{t+1}; not below the first stage).  The tile's sums go to a float accumulator with one atomic
//     add per element (vector atomics where the block is a multiple of 4 floats), laid out so
//     that a warp's additions are contiguous (acc_index).
//  2. harp_grad_theta_kernel: eight lanes per block map dL/dB to dL/dtheta in double:
//     dL/dQ = dL/dB G^T; Givens: the derivative of the rotation; Cayley: with M = (I-A)^-1
//     and Q = M (I + A), dL/dA = M^T dL/dQ (Q + I)^T and dL/dtheta_k = dL/dA[i][j] -
//     dL/dA[j][i] for the k-th pair i < j.
// The device blocks of stage 0 carry the signs (B_0 diag(S)), so kernel 1 accumulates the
// gradient of those and kernel 2 multiplies column l by the sign of its coordinate.
// Kernel 1 has 26 FMAs per byte of bf16 rows (four stages of radix 8): the FP32 pipe would bound it.  It
// runs at 27 % of the pipe's peak (65,536 rows of d = 4096: 2.82 ms; 16,384 rows from int8
// checkpoints: 0.77 ms), because a thread holds a block and its 64 sums, which leaves 8 warps per SM
// to hide the loads of tiles and blocks, the shared-memory accesses and the atomics, each of which takes a
// tenth to a fifth of the time.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "codes.cuh"
#include "harp_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTileRows = 16;

struct GradParams {
    PlanDesc pd;
    const float* lanes;                   // lane-interleaved blocks (layout in harp_internal.h)
    int64_t lane_off[HARP_MAX_STAGES];
    const void* x;
    const void* g;
    int64_t rows, ld_x, ld_g;
    float* acc;                           // dL/dB accumulators, stage t at acc + acc_off[t] (acc_index)
    int64_t acc_off[HARP_MAX_STAGES];
    int R;                                // rows per tile
    int rs;                               // row stride of the shared-memory tiles (floats)
    int64_t ntiles;
    int vec;                              // rows of x and g load as 16-byte vectors
    const float* xs;                      // x as 8-bit codes: one scale per qblock coordinates of a row
    int64_t ld_xs;
    int qshift;                           // log2 of qblock
};

// Coordinate i of a row sits at swz(i) in shared memory: bits 0-2 of i XOR bits 3-5, bits 3-4
// XOR bits 6-7.  It permutes each aligned block of 32 coordinates, and the 32 lanes of a
// warp that take 32 consecutive groups of a stage then hit 32 distinct banks for the radix
// 8, 5 and 2 stages of the workload schedules (groups of 8 contiguous coordinates, of 8
// at stride 8, and of any size at stride 64 or more).  An aligned run of 8 coordinates
// stays one aligned run of 8.
__device__ __forceinline__ int swz(int i) { return i ^ ((i >> 3) & 7) ^ (((i >> 6) & 3) << 3); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The 16 bytes of a vector load as floats (8 bf16 or 4 fp32 values).
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}

// Item q of a tile as (row r, position j of n) for q = threadIdx.x, + kThreads, ...: one division for all of them.
struct Walk {
    int r, j, dr, dj, n;
    __device__ __forceinline__ explicit Walk(int per_row) : n(per_row) {
        r = (int)threadIdx.x / n, j = (int)threadIdx.x - r * n;
        dr = kThreads / n, dj = kThreads - dr * n;
    }
    __device__ __forceinline__ void next() {
        r += dr, j += dj;
        if (j >= n) j -= n, ++r;
    }
};

// x and g rows [row0, row0 + nr) into the fp32 tiles.  Each thread keeps several loads in
// flight before it converts and stores them (a load followed directly by its store would
// wait out the memory latency once per element).
template <typename T>
__device__ void load_tile(const GradParams& p, float* A, float* H, int64_t row0, int nr) {
    const int d = (int)p.pd.d, rs = p.rs;
    const T* x = (const T*)p.x;
    const T* g = (const T*)p.g;
    if (p.vec) {
        constexpr int V = 16 / sizeof(T);   // elements per 16-byte load
        constexpr int U = 4;                // vector loads of x (and of g) in flight per thread
        const int cpr = d / V, total = nr * cpr;
        Walk from(cpr);
        for (int q0 = threadIdx.x; q0 < total; q0 += kThreads * U) {
            uint4 vx[U], vg[U];
            Walk to = from;
#pragma unroll
            for (int u = 0; u < U; ++u, from.next()) {
                const int r = from.r, j = from.j;
                if (r < nr) {
                    vx[u] = __ldg(reinterpret_cast<const uint4*>(x + (row0 + r) * p.ld_x) + j);
                    vg[u] = __ldg(reinterpret_cast<const uint4*>(g + (row0 + r) * p.ld_g) + j);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u, to.next()) {
                const int r = to.r, j = to.j;
                if (r < nr) {
                    float fx[V], fg[V];
                    unpack(vx[u], fx);
                    unpack(vg[u], fg);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        A[r * rs + swz(j * V + e)] = fx[e];
                        H[r * rs + swz(j * V + e)] = fg[e];
                    }
                }
            }
        }
    } else {
        constexpr int U = 8;
        const int total = nr * d;
        for (int q0 = threadIdx.x; q0 < total; q0 += kThreads * U) {
            float fx[U], fg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kThreads;
                if (q < total) {
                    const int r = q / d, i = q - r * d;
                    fx[u] = to_f32(__ldg(x + (row0 + r) * p.ld_x + i));
                    fg[u] = to_f32(__ldg(g + (row0 + r) * p.ld_g + i));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kThreads;
                if (q < total) {
                    const int r = q / d, i = q - r * d;
                    A[r * rs + swz(i)] = fx[u];
                    H[r * rs + swz(i)] = fg[u];
                }
            }
        }
    }
}

// The same for rows of x that are kept as 8-bit codes of format C: x^ = code * scale, rounded to
// fp32.  A thread takes 8 coordinates (one scale) of a row at a time; vec: 8-byte loads of codes and
// 16-byte loads of g.
template <typename C, typename T>
__device__ void load_tile_codes(const GradParams& p, float* A, float* H, int64_t row0, int nr) {
    const int d = (int)p.pd.d, rs = p.rs;
    const uint8_t* x = (const uint8_t*)p.x;
    const T* g = (const T*)p.g;
    constexpr int U = 4;                // groups of 8 in flight per thread
    const int cpr = (d + 7) / 8, total = nr * cpr;
    Walk from(cpr);
    auto put = [&](int r, int c, const uint2& code, float s, const float (&fg)[8]) {
        const int n = min(8, d - c);
        float lo[4], hi[4];
        C::decode4(code.x, lo);
        C::decode4(code.y, hi);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k < n) {
                A[r * rs + swz(c + k)] = (k < 4 ? lo[k & 3] : hi[k & 3]) * s;
                H[r * rs + swz(c + k)] = fg[k];
            }
        }
    };
    if (p.vec && (d & 7) == 0) {
        for (int q0 = threadIdx.x; q0 < total; q0 += kThreads * U) {
            uint2 code[U];
            float s[U];
            harp_codes::Eight<T> g8[U];
            Walk to = from;
#pragma unroll
            for (int u = 0; u < U; ++u, from.next()) {
                const int r = from.r, c = 8 * from.j;
                if (r < nr) {
                    code[u] = __ldcs(reinterpret_cast<const uint2*>(x + (row0 + r) * p.ld_x + c));
                    s[u] = __ldg(p.xs + (row0 + r) * p.ld_xs + (c >> p.qshift));
                    g8[u].load(g + (row0 + r) * p.ld_g + c);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u, to.next()) {
                float fg[8];
                g8[u].get(fg);
                if (to.r < nr) put(to.r, 8 * to.j, code[u], s[u], fg);
            }
        }
    } else {
        for (; from.r < nr; from.next()) {
            const int r = from.r, c = 8 * from.j, n = min(8, d - c);
            const uint8_t* src = x + (row0 + r) * p.ld_x + c;
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) w[k >> 2] |= (uint32_t)src[k] << (8 * (k & 3));
            float fg[8];
            harp_codes::load8(g + (row0 + r) * p.ld_g + c, n, false, fg);
            put(r, c, make_uint2(w[0], w[1]), __ldg(p.xs + (row0 + r) * p.ld_xs + (c >> p.qshift)), fg);
        }
    }
}

// Block c of a stage from the lane-interleaved copy: B[k][l] -> w[k * B + l].
template <int B>
__device__ __forceinline__ void load_block(const float* lanes, int64_t c, float (&w)[B * B]) {
    constexpr int BB = B * B;
    const int64_t grp = c >> 5, lane = c & 31;
    if constexpr (BB % 4 == 0) {
        const float4* p = reinterpret_cast<const float4*>(lanes) + grp * (BB / 4) * 32 + lane;
#pragma unroll
        for (int j = 0; j < BB / 4; ++j) {
            const float4 v = __ldg(p + j * 32);
            w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
    } else {
        const float* p = lanes + grp * BB * 32 + lane;
#pragma unroll
        for (int e = 0; e < BB; ++e) w[e] = __ldg(p + e * 32);
    }
}

// Entry e of block c in a stage's accumulator: like the lane-interleaved blocks (groups of 32 blocks, 16-byte
// pieces or floats of a group's blocks side by side), so that a warp's atomic additions cover contiguous
// bytes; the blocks behind the last whole group lie one after the other, and the size stays the blocks'.
template <int BB>
__device__ __forceinline__ int64_t acc_index(int64_t c, int e, int64_t nb) {
    const int64_t grp = c >> 5, lane = c & 31;
    if (c >= (nb & ~(int64_t)31)) return c * BB + e;
    if (BB % 4 == 0) return ((grp * (BB / 4) + (e >> 2)) * 32 + lane) * 4 + (e & 3);
    return (grp * BB + e) * 32 + lane;
}
__device__ __forceinline__ int64_t acc_index(int bb, int64_t c, int e, int64_t nb) {
    const int64_t grp = c >> 5, lane = c & 31;
    if (c >= (nb & ~(int64_t)31)) return c * bb + e;
    if (bb % 4 == 0) return ((grp * (bb / 4) + (e >> 2)) * 32 + lane) * 4 + (e & 3);
    return (grp * bb + e) * 32 + lane;
}

// Two fp32 values in one register pair: a b + c for both with one instruction (each rounded to nearest).
// The backward stages take pairs of neighbouring columns (16,384 rows of d = 4096: 0.81 -> 0.77 ms; the
// forward stage in pairs: 0.78).
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Forward stage t on the activation tile: z <- M_t z.
template <int B>
__device__ void stage_forward(float* A, int nr, int rs, int nb, int s, const float* lanes) {
    for (int c = threadIdx.x; c < nb; c += kThreads) {
        float w[B * B];
        load_block<B>(lanes, c, w);
        const int hi = (unsigned)c / (unsigned)s, lo = c - hi * s;
        int off[B];
#pragma unroll
        for (int k = 0; k < B; ++k) off[k] = swz(lo + s * (k + B * hi));
        for (int r = 0; r < nr; ++r) {
            float* a = A + r * rs;
            float xv[B];
#pragma unroll
            for (int l = 0; l < B; ++l) xv[l] = a[off[l]];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                float acc = 0.f;
#pragma unroll
                for (int l = 0; l < B; ++l) acc = fmaf(w[k * B + l], xv[l], acc);
                a[off[k]] = acc;
            }
        }
    }
}

// Backward stage t: with z = z_{t+1} in A and h = h_{t+1} in H, per group and row
//   z_t = B^T z,  dL/dB += h z_t^T,  h_t = B^T h,
// then the tile's sums of this group go to the accumulator.  The last stage is not run forward, A still
// holds its z_t; nothing reads the first stage's h_t and, behind it, A.
enum Place { kMiddle, kLast, kFirst };
template <int B, Place AT>
__device__ void stage_backward(float* A, float* H, int nr, int rs, int nb, int s, const float* lanes,
                               float* acc_t) {
    constexpr int BB = B * B;
    for (int c = threadIdx.x; c < nb; c += kThreads) {
        float w[BB];
        load_block<B>(lanes, c, w);
        const int hi = (unsigned)c / (unsigned)s, lo = c - hi * s;
        int off[B];
#pragma unroll
        for (int k = 0; k < B; ++k) off[k] = swz(lo + s * (k + B * hi));
        float sum[BB];
        if constexpr (B % 2 == 0) {
            uint64_t acc[BB / 2];   // pairs of neighbouring columns
#pragma unroll
            for (int e = 0; e < BB / 2; ++e) acc[e] = 0;
            for (int r = 0; r < nr; ++r) {
                float* a = A + r * rs;
                float* h = H + r * rs;
                float zf[B];
                uint64_t zo[B], ho[B];
#pragma unroll
                for (int k = 0; k < B; ++k) {
                    const float hf = h[off[k]];
                    zf[k] = a[off[k]];
                    zo[k] = pair2(zf[k], zf[k]), ho[k] = pair2(hf, hf);
                }
#pragma unroll
                for (int l = 0; l < B; l += 2) {
                    uint64_t zi = 0, hin = 0;
                    if (AT == kLast) zi = pair2(zf[l], zf[l + 1]);
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        const uint64_t w2 = pair2(w[k * B + l], w[k * B + l + 1]);
                        if (AT != kLast) zi = fma2(w2, zo[k], zi);
                        if (AT != kFirst) hin = fma2(w2, ho[k], hin);
                    }
#pragma unroll
                    for (int k = 0; k < B; ++k) acc[(k * B + l) / 2] = fma2(ho[k], zi, acc[(k * B + l) / 2]);
                    if (AT == kMiddle) split2(zi, a[off[l]], a[off[l + 1]]);
                    if (AT != kFirst) split2(hin, h[off[l]], h[off[l + 1]]);
                }
            }
#pragma unroll
            for (int e = 0; e < BB / 2; ++e) split2(acc[e], sum[2 * e], sum[2 * e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < BB; ++e) sum[e] = 0.f;
            for (int r = 0; r < nr; ++r) {
                float* a = A + r * rs;
                float* h = H + r * rs;
                float zo[B], ho[B];
#pragma unroll
                for (int k = 0; k < B; ++k) zo[k] = a[off[k]], ho[k] = h[off[k]];
#pragma unroll
                for (int l = 0; l < B; ++l) {
                    float zi = AT == kLast ? zo[l] : 0.f, hin = 0.f;
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        if (AT != kLast) zi = fmaf(w[k * B + l], zo[k], zi);
                        if (AT != kFirst) hin = fmaf(w[k * B + l], ho[k], hin);
                    }
#pragma unroll
                    for (int k = 0; k < B; ++k) sum[k * B + l] = fmaf(ho[k], zi, sum[k * B + l]);
                    if (AT == kMiddle) a[off[l]] = zi;
                    if (AT != kFirst) h[off[l]] = hin;
                }
            }
        }
        float* dst = acc_t + acc_index<BB>(c, 0, nb);
        const int step = c < (nb & ~(int64_t)31) ? (BB % 4 == 0 ? 128 : 32) : (BB % 4 == 0 ? 4 : 1);
        if constexpr (BB % 4 == 0) {
#pragma unroll
            for (int e = 0; e < BB; e += 4)
                atomicAdd(reinterpret_cast<float4*>(dst + e / 4 * step), make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]));
        } else {
#pragma unroll
            for (int e = 0; e < BB; ++e) atomicAdd(dst + e * step, sum[e]);
        }
    }
}

template <bool FWD>
__device__ void run_stage(const GradParams& p, int t, float* A, float* H, int nr) {
    const StageDesc& sd = p.pd.st[t];
    const float* lanes = p.lanes + p.lane_off[t];
    const int s = (int)sd.s;
    const int nb = (int)sd.nblocks;
    float* acc_t = p.acc + p.acc_off[t];
#define HARP_GRAD_CASE(BV)                                                                                     \
    case BV:                                                                                                   \
        if (FWD) stage_forward<BV>(A, nr, p.rs, nb, s, lanes);                                                 \
        else if (t == 0) stage_backward<BV, kFirst>(A, H, nr, p.rs, nb, s, lanes, acc_t);                      \
        else if (t == p.pd.m - 1) stage_backward<BV, kLast>(A, H, nr, p.rs, nb, s, lanes, acc_t);              \
        else stage_backward<BV, kMiddle>(A, H, nr, p.rs, nb, s, lanes, acc_t);                                 \
        break;
    switch (sd.b) {
        HARP_GRAD_CASE(2)
        HARP_GRAD_CASE(3)
        HARP_GRAD_CASE(4)
        HARP_GRAD_CASE(5)
        HARP_GRAD_CASE(6)
        HARP_GRAD_CASE(7)
        HARP_GRAD_CASE(8)
        default: break;
    }
#undef HARP_GRAD_CASE
    __syncthreads();
}

// C: void for rows of x in the type of g, else the format of their 8-bit codes.
template <typename T, typename C = void>
__global__ void __launch_bounds__(kThreads, 1) harp_grad_blocks_kernel(const __grid_constant__ GradParams p) {
    extern __shared__ __align__(16) float smem[];
    float* A = smem;                   // activations [row][swz(i)]
    float* H = smem + p.R * p.rs;      // gradients   [row][swz(i)]
    const int m = p.pd.m;
    for (int64_t tile = blockIdx.x; tile < p.ntiles; tile += gridDim.x) {
        const int64_t row0 = tile * p.R;
        const int nr = (int)min((int64_t)p.R, p.rows - row0);
        if constexpr (std::is_void<C>::value) load_tile<T>(p, A, H, row0, nr);
        else load_tile_codes<C, T>(p, A, H, row0, nr);
        __syncthreads();
        for (int t = 0; t < max(1, m - 1); ++t) run_stage<true>(p, t, A, H, nr);
        for (int t = m - 1; t >= 0; --t) run_stage<false>(p, t, A, H, nr);
    }
}

struct StageOffsets {
    int64_t off[HARP_MAX_STAGES];
};

// dL/dB -> dL/dtheta in double, eight lanes per block: lane i holds row i of every matrix in
// registers, and rows go round by shuffles (one thread per block, its matrices in local memory, took
// 0.12 ms whatever the batch).
__global__ void harp_grad_theta_kernel(PlanDesc pd, const float* __restrict__ theta_f32,
                                       const int8_t* __restrict__ theta_i8, const float* __restrict__ scales,
                                       const double* __restrict__ mixers, const int8_t* __restrict__ signs,
                                       const float* __restrict__ acc, StageOffsets acc_off,
                                       float* __restrict__ dtheta, int64_t total_blocks) {
    const int64_t gid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 3;
    const int i = threadIdx.x & 7;                  // this lane's row
    const bool live = gid < total_blocks;
    int t = 0;
    int64_t c = live ? gid : 0;
    while (t < pd.m - 1 && c >= pd.st[t].nblocks) {
        c -= pd.st[t].nblocks;
        ++t;
    }
    const StageDesc sd = pd.st[t];
    const int b = sd.b;
    const int64_t poff = sd.theta_off + c * sd.p;
    const double scale = theta_i8 ? (double)scales[t] : 1.0;
    auto param = [&](int k) -> double {
        return theta_i8 ? (double)theta_i8[poff + k] * scale : (double)theta_f32[poff + k];
    };
    const float* pb = acc + acc_off.off[t];
    const double* gm = mixers + sd.mixer_off;
    // R = dL/dB G^T, with stage 0's sign on column l (the device blocks are B_0 diag(S)); rows and
    // columns from b on are zero
    double row[8], R[8];
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        double v = i < b && l < b ? (double)pb[acc_index(b * b, c, i * b + l, sd.nblocks)] : 0.0;
        if (t == 0 && l < b && signs[l + b * c] < 0) v = -v;
        row[l] = v;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        double v = 0.0;
#pragma unroll
        for (int l = 0; l < 8; ++l)
            if (j < b && l < b) v += row[l] * gm[j * b + l];
        R[j] = v;
    }
    float* out = dtheta + poff;
    const unsigned all = 0xffu << (threadIdx.x & 24);   // this block's lanes, which take the same branches
    if (b == 2) {
        const double th = param(0), cs = cos(th), sn = sin(th);
        const double r10 = __shfl_sync(all, R[0], 1, 8), r11 = __shfl_sync(all, R[1], 1, 8);
        if (live && i == 0) out[0] = (float)(-R[0] * sn - R[1] * cs + r10 * cs - r11 * sn);
        return;
    }
    // M = (I - A)^{-1} by Gauss-Jordan without pivoting (every leading principal minor of
    // I - A, A skew, is a product of (1 + lambda^2) > 0), then Q = M (I + A).  Rows from b on: identity.
    double lhs[8], M[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lhs[j] = M[j] = i == j ? 1.0 : 0.0;
        if (i != j && i < b && j < b) {
            const int lo = min(i, j), hi = max(i, j);
            const double a = param(lo * b - lo * (lo + 1) / 2 + hi - lo - 1);   // pair (lo, hi) of the upper triangle
            lhs[j] = i < j ? -a : a;
        }
    }
#pragma unroll
    for (int col = 0; col < 8; ++col) {
        const double inv = 1.0 / __shfl_sync(all, lhs[col], col, 8);
        const double f = lhs[col];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double pl = __shfl_sync(all, lhs[j], col, 8) * inv, pm = __shfl_sync(all, M[j], col, 8) * inv;
            if (i == col) {
                lhs[j] = pl, M[j] = pm;
            } else {
                lhs[j] -= f * pl, M[j] -= f * pm;
            }
        }
    }
    // I + A = 2 I - (I - A); Q = M (I + A) = 2 M - I
    // E = M^T R (Q + I)^T = M^T R (2 M)^T: T1 = M^T R first, lane i its row i
    double T1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) T1[j] = 0.0;
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        double mli = 0.0;   // M[l][i]
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double v = __shfl_sync(all, M[j], l, 8);
            if (j == i) mli = v;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) T1[j] += mli * __shfl_sync(all, R[j], l, 8);
    }
    double E[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        double v = 0.0;
#pragma unroll
        for (int l = 0; l < 8; ++l) {
            const double q = 2.0 * __shfl_sync(all, M[l], j, 8) - (j == l ? 1.0 : 0.0);   // Q[j][l]
            if (l < b) v += T1[l] * (q + (j == l ? 1.0 : 0.0));
        }
        E[j] = v;
    }
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        // E[i][j] - E[j][i] for i < j: lane j hands over its E[i], a register that depends on the lane
        double other = 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double v = __shfl_sync(all, E[k], j, 8);
            if (k == i) other = v;
        }
        if (live && i < j && j < b) out[i * b - i * (i + 1) / 2 + j - i - 1] = (float)(E[j] - other);
    }
}

int sms_of_current_device() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = 1;
    }
    return n;
}

// Accumulators: per stage nblocks * b * b floats, each stage starting on a 16-byte
// boundary (vector atomics).
struct AccLayout {
    StageOffsets off = {};
    int64_t floats = 0;          // accumulator floats
    size_t bytes = 0;            // workspace bytes
};

AccLayout acc_layout(const PlanDesc& pd) {
    AccLayout L;
    int64_t off = 0;
    for (int t = 0; t < pd.m; ++t) {
        L.off.off[t] = off;
        off += (pd.st[t].nblocks * pd.st[t].b * pd.st[t].b + 3) / 4 * 4;
    }
    L.floats = off;
    L.bytes = (size_t)off * 4;
    return L;
}

}  // namespace

extern "C" size_t harp_grad_workspace_bytes(harp_plan_t p) {
    if (!p) return 0;
    return acc_layout(p->desc).bytes;
}

namespace {

// Rows of x as 8-bit codes; scales == NULL: rows of x in the type of g.
struct CodedRows {
    harp_code code;
    const float* scales;
    int64_t ld_s;
    int qblock;
};

template <typename T, typename C>
cudaError_t launch_blocks(const GradParams& gp, int grid, size_t smem, cudaStream_t s) {
    const cudaError_t e = (cudaError_t)harp_set_smem_limit((const void*)harp_grad_blocks_kernel<T, C>, (int)smem);
    if (e != cudaSuccess) return e;
    harp_grad_blocks_kernel<T, C><<<grid, kThreads, smem, s>>>(gp);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_blocks(const GradParams& gp, const CodedRows& cr, int grid, size_t smem, cudaStream_t s) {
    if (!cr.scales) return launch_blocks<T, void>(gp, grid, smem, s);
    return cr.code == HARP_CODE_I8 ? launch_blocks<T, harp_codes::CodeI8>(gp, grid, smem, s)
                                   : launch_blocks<T, harp_codes::CodeE4M3>(gp, grid, smem, s);
}

harp_status grad_checked(harp_plan_t p, const void* x, const void* g, int64_t rows, int64_t ld_x, int64_t ld_g,
                         harp_dtype dtype, const CodedRows& cr, bool coded, float* dtheta, void* workspace,
                         size_t ws_bytes, void* stream) {
    if (!p) return harp_fail(HARP_ERR_INVALID_ARG, "plan is NULL");
    if (dtype != HARP_F32 && dtype != HARP_BF16) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown dtype");
    if (rows < 0) return harp_fail(HARP_ERR_INVALID_ARG, "rows < 0");
    const PlanDesc& pd = p->desc;
    const int64_t d = pd.d;
    if (ld_x < d || ld_g < d) return harp_fail(HARP_ERR_INVALID_ARG, "leading dimension smaller than d");
    if (!dtheta) return harp_fail(HARP_ERR_INVALID_ARG, "dtheta is NULL");
    if (p->composite) return harp_fail(HARP_ERR_UNSUPPORTED, "the gradient is taken for one plan, not a composite");
    {
        const harp_status mst = harp_require_materialized(p, stream);
        if (mst != HARP_OK) return mst;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return harp_fail(HARP_ERR_CUDA, "no CUDA device");
    }
    if (dev != p->device) return harp_fail(HARP_ERR_WRONG_DEVICE, "plan materialized on another device");
    for (int t = 0; t < pd.m; ++t)
        if (pd.st[t].b > 8) return harp_fail(HARP_ERR_UNSUPPORTED, "the gradient kernel takes radices up to 8");
    const AccLayout L = acc_layout(pd);
    if (!workspace || ws_bytes < L.bytes)
        return harp_fail(HARP_ERR_INVALID_ARG, "workspace smaller than harp_grad_workspace_bytes()");
    if (((uintptr_t)workspace & 15) != 0) return harp_fail(HARP_ERR_INVALID_ARG, "workspace not 16-byte aligned");
    if (rows > 0 && (!x || !g)) return harp_fail(HARP_ERR_INVALID_ARG, "x or g is NULL");
    if (rows > 0 && coded && !cr.scales) return harp_fail(HARP_ERR_INVALID_ARG, "the codes' scales are NULL");
    {
        // the accumulators are zeroed and then added to while x and g are read, and dtheta is
        // written last: none of them may share memory with another
        const size_t es = dtype == HARP_F32 ? 4 : 2;
        const size_t xb = rows > 0 ? ((size_t)(rows - 1) * ld_x + d) * (coded ? 1 : es) : 0;
        const size_t gb = rows > 0 ? ((size_t)(rows - 1) * ld_g + d) * es : 0;
        const size_t tb = (size_t)p->theta_total * sizeof(float);
        if (rows > 0 && (ranges_overlap(workspace, ws_bytes, x, xb) || ranges_overlap(workspace, ws_bytes, g, gb)))
            return harp_fail(HARP_ERR_INVALID_ARG, "workspace overlaps x or g");
        if (ranges_overlap(dtheta, tb, workspace, ws_bytes) ||
            (rows > 0 && (ranges_overlap(dtheta, tb, x, xb) || ranges_overlap(dtheta, tb, g, gb))))
            return harp_fail(HARP_ERR_INVALID_ARG, "dtheta overlaps the workspace, x or g");
        if (rows > 0 && coded) {
            const size_t sb = ((size_t)(rows - 1) * cr.ld_s + (d + cr.qblock - 1) / cr.qblock) * sizeof(float);
            if (ranges_overlap(workspace, ws_bytes, cr.scales, sb) || ranges_overlap(dtheta, tb, cr.scales, sb))
                return harp_fail(HARP_ERR_INVALID_ARG, "dtheta or the workspace overlaps the scales");
        }
    }
    // rows per tile: two fp32 tiles of rows rounded up to 32 coordinates (the swizzle
    // permutes aligned blocks of 32) within the 227 KiB of shared memory a CTA may use
    const int rs = (int)((d + 31) / 32 * 32);
    const int64_t per_row = 2 * (int64_t)rs * 4;
    const int64_t budget = 227 * 1024;
    int R = (int)std::min<int64_t>(kMaxTileRows, budget / per_row);
    if (R >= 1 && rows > 0) {
        // the same number of rounds over the SMs in tiles as low as they may be: no SM waits for another's
        // full tile (1,001 rows of d = 5120: two rounds of 4 rows instead of 5)
        const int64_t sms = sms_of_current_device(), rounds = (rows + R * sms - 1) / (R * sms);
        R = (int)((rows + rounds * sms - 1) / (rounds * sms));
    }
    if (R < 1) return harp_fail(HARP_ERR_UNSUPPORTED, "a row is too long for the gradient kernel's tile");

    cudaStream_t s = (cudaStream_t)stream;
    float* acc = (float*)workspace;
    cudaError_t e = cudaMemsetAsync(acc, 0, (size_t)L.floats * 4, s);
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    if (rows > 0) {
        GradParams gp;
        gp.pd = pd;
        gp.lanes = p->d_blocks_lanes;
        for (int t = 0; t < HARP_MAX_STAGES; ++t) gp.lane_off[t] = p->lane_off[t], gp.acc_off[t] = L.off.off[t];
        gp.x = x;
        gp.g = g;
        gp.rows = rows;
        gp.ld_x = ld_x;
        gp.ld_g = ld_g;
        gp.acc = acc;
        gp.R = R;
        gp.rs = rs;
        gp.ntiles = (rows + R - 1) / R;
        const size_t es = dtype == HARP_F32 ? 4 : 2;
        gp.xs = cr.scales, gp.ld_xs = cr.ld_s;
        gp.qshift = cr.qblock == 32 ? 5 : cr.qblock == 64 ? 6 : cr.qblock == 128 ? 7 : 8;
        const bool one = rows == 1;   // a single row is never stepped past
        if (coded)
            gp.vec = ((uintptr_t)x % 8 == 0) && ((uintptr_t)g % 16 == 0) && (one || (ld_x % 8 == 0 && (ld_g * es) % 16 == 0));
        else
            gp.vec = ((uintptr_t)x % 16 == 0) && ((uintptr_t)g % 16 == 0) &&
                     (one || ((ld_x * es) % 16 == 0 && (ld_g * es) % 16 == 0)) && (d * es) % 16 == 0;
        const size_t smem = (size_t)R * per_row;
        const int grid = (int)std::min<int64_t>(gp.ntiles, sms_of_current_device());
        e = dtype == HARP_BF16 ? launch_blocks<__nv_bfloat16>(gp, cr, grid, smem, s)
                               : launch_blocks<float>(gp, cr, grid, smem, s);
        if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    }
    int64_t total = 0;
    for (int t = 0; t < pd.m; ++t) total += pd.st[t].nblocks;
    const bool i8 = p->kind == HARP_THETA_I8;
    harp_grad_theta_kernel<<<(unsigned)((8 * total + 127) / 128), 128, 0, s>>>(
        pd, i8 ? nullptr : (const float*)p->d_theta, i8 ? (const int8_t*)p->d_theta : nullptr, p->d_scales,
        p->d_mixers, p->d_signs, acc, L.off, dtheta, total);
    e = cudaGetLastError();
    if (e != cudaSuccess) return harp_fail(HARP_ERR_CUDA, cudaGetErrorString(e));
    harp_set_last_kernel("harp_grad_blocks_kernel");
    return HARP_OK;
}

}  // namespace

extern "C" harp_status harp_grad_theta(harp_plan_t p, const void* x, const void* g, int64_t rows, int64_t ld_x,
                                       int64_t ld_g, harp_dtype dtype, float* dtheta, void* workspace,
                                       size_t ws_bytes, void* stream) {
    harp_clear_error();
    return grad_checked(p, x, g, rows, ld_x, ld_g, dtype, CodedRows{HARP_CODE_I8, nullptr, 0, 1}, false, dtheta,
                        workspace, ws_bytes, stream);
}

extern "C" harp_status harp_grad_theta_quant(harp_plan_t p, const void* q, int64_t ld_q, harp_code code,
                                             const float* scales, int64_t ld_s, int32_t qblock, const void* g,
                                             int64_t ld_g, harp_dtype dtype, int64_t rows, float* dtheta,
                                             void* workspace, size_t ws_bytes, void* stream) {
    harp_clear_error();
    if (!p) return harp_fail(HARP_ERR_INVALID_ARG, "plan is NULL");
    if (code != HARP_CODE_I8 && code != HARP_CODE_E4M3) return harp_fail(HARP_ERR_UNSUPPORTED, "unknown code format");
    if (qblock != 32 && qblock != 64 && qblock != 128 && qblock != 256)
        return harp_fail(HARP_ERR_INVALID_ARG, "qblock must be 32, 64, 128 or 256");
    if (ld_s < (p->desc.d + qblock - 1) / qblock)
        return harp_fail(HARP_ERR_INVALID_ARG, "leading dimension smaller than the row");
    if ((uintptr_t)scales % 4 || (uintptr_t)g % (dtype == HARP_F32 ? 4 : 2))
        return harp_fail(HARP_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    return grad_checked(p, q, g, rows, ld_q, ld_g, dtype, CodedRows{code, scales, ld_s, qblock}, true, dtheta,
                        workspace, ws_bytes, stream);
}
