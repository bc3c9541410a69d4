// Instantiations of the cluster row kernel for bf16 rows in and e4m3 codes with per-block scales out
// (the fused quantizer), for the inverse.
#include <cuda_bf16.h>

#include "apply_cluster.cuh"

cudaError_t harp_cluster_launch_bf16_e4m3(int which, int cl, const harp_cluster::ClusterParams& cp, size_t smem, int grid,
                                          cudaStream_t stream) {
    return harp_cluster::launch_mask<__nv_bfloat16, __nv_fp8_e4m3, true, 0>(which, cl, cp, smem, grid, stream);
}
