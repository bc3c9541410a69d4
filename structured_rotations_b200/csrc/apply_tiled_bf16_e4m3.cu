// Instantiations of the tiled row kernel for bf16 rows in and e4m3 codes with per-block
// fp32 scales out (the fused quantizer epilogue).
#include <cuda_bf16.h>

#include "apply_tiled.cuh"

cudaError_t harp_tiled_launch_bf16_e4m3(int which, int V, int nt, int cl, bool inverse,
                                        const harp_tiled::TiledParams& tp, size_t smem, int grid, cudaStream_t stream) {
    return harp_tiled::launch<__nv_bfloat16, __nv_fp8_e4m3>(which, V, nt, cl, inverse, tp, smem, grid, stream);
}
