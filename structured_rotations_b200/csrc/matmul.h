// The e4m3 product's operands and helpers, shared by its kernels (matmul.cu, matmul_rows.cu,
// matmul_tiles.cu).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "harp.h"
#include "tc.cuh"

struct MatmulParams {
    const uint8_t *x, *w;        // codes: rows x k, n x k
    const float *sx, *sw;        // scales: rows x kb, ceil(n / 128) x kb
    void* y;                     // rows x n
    int64_t ld_x, ld_w, ld_sx, ld_sw, ld_y;
    int64_t rows, n, k, kb;      // kb: blocks of 128 along k, the last one possibly short
};

// The factor sx sw of a block's sum S (zero, or 2^-18 <= |S| < 2^25).  Scales span 2^-109 to 2^119, so that their
// fp32 product may underflow or overflow where S sx sw does neither, or where S is zero.  Then S meets them one
// after the other, (S first) second: the larger one first where the product is too small (S first is
// below 2^48 then), the smaller one where it is too large (S first is above 2^-20 then, and overflows only
// with the result).  Else first = 1 and second is the product.  A zero scale needs no care, and a NaN stays one.
__device__ __forceinline__ bool scales_apart(float sx, float sw) {
    const float m = fabsf(sx * sw);
    return !(m >= 1.17549435e-38f && m <= 3.40282347e38f) && sx != 0.f && sw != 0.f;   // 2^-126, the largest finite value
}
// the product, or a NaN in the place of one that cannot stand for its scales
__device__ __forceinline__ float factor_or_nan(float sx, float sw) {
    return scales_apart(sx, sw) ? __int_as_float(0x7fffffff) : sx * sw;
}
struct BlockFactor {
    float first, second;
};
__device__ __forceinline__ BlockFactor block_factor(float sx, float sw) {
    if (!scales_apart(sx, sw)) return {1.f, sx * sw};
    const bool x_first = (fabsf(sx) > fabsf(sw)) == (fabsf(sx * sw) < 1.f);
    return {x_first ? sx : sw, x_first ? sw : sx};
}

// Map of a matrix of codes in boxes of 128 bytes x `box` rows, 128-byte swizzled; beyond the matrix the
// boxes hold zeros (matmul.cu).
harp_status matmul_tensor_map(CUtensorMap* map, const void* q, int64_t rows, int64_t k, int64_t ld, int box);
// The current device's status word of bounded waits (nullptr: no address); see harp_device_status.
int* matmul_status_word();
// The limit of this host thread's next launches (tc.cuh; harp_test_inject_wait_timeout).
harp_tc::WaitLimit matmul_wait_limit();

// Few rows (at most 128): 16-byte aligned operands and leading dimensions.
harp_status launch_matmul_rows(const MatmulParams& p, harp_dtype out, void* stream);
// Many rows: the same alignment.
harp_status launch_matmul_tiles(const MatmulParams& p, harp_dtype out, void* stream);
