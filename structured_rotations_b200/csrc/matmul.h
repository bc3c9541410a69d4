// The e4m3 product's operands and helpers, shared by its kernels (matmul.cu, matmul_rows.cu,
// matmul_tiles.cu).
#pragma once

#include <cstdint>

#include <cuda.h>

#include "harp.h"

struct MatmulParams {
    const uint8_t *x, *w;        // codes: rows x k, n x k
    const float *sx, *sw;        // scales: rows x kb, ceil(n / 128) x kb
    void* y;                     // rows x n
    int64_t ld_x, ld_w, ld_sx, ld_sw, ld_y;
    int64_t rows, n, k, kb;      // kb: blocks of 128 along k, the last one possibly short
};

// Map of a matrix of codes in boxes of 128 bytes x `box` rows, 128-byte swizzled; beyond the matrix the
// boxes hold zeros (matmul.cu).
harp_status matmul_tensor_map(CUtensorMap* map, const void* q, int64_t rows, int64_t k, int64_t ld, int box);
// The current device's status word of bounded waits (nullptr: no address); see harp_device_status.
int* matmul_status_word();

// Few rows: 16-byte aligned operands and leading dimensions.
harp_status launch_matmul_rows(const MatmulParams& p, harp_dtype out, void* stream);
// Many rows: the same alignment.
harp_status launch_matmul_tiles(const MatmulParams& p, harp_dtype out, void* stream);
