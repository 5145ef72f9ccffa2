// kda_norm_quant of fp32 rows: a translation unit per type, compiled in parallel.
#include "kda_norm_quant.cuh"

namespace kda {

cudaError_t launch_norm_quant_fp32(const NormQuantParams &p, cudaStream_t stream) { return by_alignment<Fp32>(p, stream); }

}  // namespace kda
