// kda_norm_quant of bf16 rows (and the choice by type): a translation unit per type, compiled in parallel.
#include "kda_norm_quant.cuh"

namespace kda {

cudaError_t launch_norm_quant_bf16(const NormQuantParams &p, cudaStream_t stream) { return by_alignment<Bf16>(p, stream); }

cudaError_t launch_norm_quant(const NormQuantParams &p, int dtype, cudaStream_t stream)
{
    return dtype == 0 ? launch_norm_quant_bf16(p, stream) : dtype == 1 ? launch_norm_quant_fp16(p, stream) : launch_norm_quant_fp32(p, stream);
}

}  // namespace kda
