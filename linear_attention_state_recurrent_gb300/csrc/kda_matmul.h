// Internal parameters and launchers of the 16-bit matrix product, shared by its entry points and kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct MatmulParams {
    const void *a;      int64_t ld_a;
    const void *w;      int64_t ld_w;
    int M, N, K;
    const void *bias;   int bias_dtype;     // a's type or fp32; NULL: none
    int act;                                // KDA_ACT_*
    const void *res;    int64_t ld_res;     // out's type; NULL: none
    void *out;          int64_t ld_out;
    int dtype, out_dtype;
    uint32_t *err;
};

cudaError_t launch_matmul(const MatmulParams &p, cudaStream_t stream);
// Rows of a per tile (0: operands off 16-byte boundaries), CTAs that split the inner axis.
cudaError_t plan_matmul(const MatmulParams &p, int32_t (&plan)[2]);

}  // namespace kda
