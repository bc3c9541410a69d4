// The e4m3 product's operands, shared by its kernels (matmul.cu).
#pragma once

#include <cstdint>

struct MatmulParams {
    const uint8_t *x, *w;        // codes: rows x k, n x k
    const float *sx, *sw;        // scales: rows x kb, ceil(n / 128) x kb
    void* y;                     // rows x n
    int64_t ld_x, ld_w, ld_sx, ld_sw, ld_y;
    int64_t rows, n, k, kb;      // kb: blocks of 128 along k, the last one possibly short
};
