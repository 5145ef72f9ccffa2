// kda_fp8_matmul: out = A W^T with e4m3 operands and a scale for each block of 128.
#include <climits>
#include <cstdint>
#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_layer.h"
#include "kda_pdl.cuh"

namespace kda {
namespace {

// e4m3 -> fp32 (exact)
__device__ __forceinline__ float e4m3_to_f32(uint8_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

__device__ __forceinline__ void store_out(void *out, int64_t i, int dtype, float v)
{
    if (dtype == 0) static_cast<uint16_t *>(out)[i] = f32_to_bf16(v);
    else if (dtype == 1) static_cast<__half *>(out)[i] = __float2half_rn(v);
    else static_cast<float *>(out)[i] = v;
}

// Any strides and alignments: 64 x 64 tiles on the ordinary FMA units.
constexpr int GT = 64, GK = 32;
__global__ void __launch_bounds__(256) fp8_general_kernel(const Fp8Params p, int tiles_n)
{
    __shared__ float sA[GK][GT + 1], sB[GK][GT + 1];
    pdl_wait_then_release();
    const int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
    const int64_t m0 = static_cast<int64_t>(tm) * GT, n0 = static_cast<int64_t>(tn) * GT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int g = 0; g * 128 < p.K; g++) {
        float part[4][4] = {};
        for (int k0 = g * 128; k0 < g * 128 + 128 && k0 < p.K; k0 += GK) {
            __syncthreads();
            for (int i = threadIdx.x; i < GT * GK; i += 256) {
                const int row = i / GK, k = i % GK;
                const bool in = k0 + k < p.K;
                sA[k][row] = in && m0 + row < p.M ? e4m3_to_f32(p.a[(m0 + row) * p.ld_a + k0 + k]) : 0.f;
                sB[k][row] = in && n0 + row < p.N ? e4m3_to_f32(p.w[(n0 + row) * p.ld_w + k0 + k]) : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < GK; k++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) part[i][j] = fmaf(sA[k][ty + 16 * i], sB[k][tx + 16 * j], part[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t m = m0 + ty + 16 * i;
            if (m >= p.M) continue;
            const float sa = p.sa[m * p.sa_row + g * p.sa_group];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int64_t n = n0 + tx + 16 * j;
                if (n < p.N) acc[i][j] = fmaf(part[i][j], sa * p.sw[(n / 128) * p.sw_row + g * p.sw_group], acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) store_out(p.out, m * p.ld_out + n, p.out_dtype, acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Params &p, cudaStream_t stream)
{
    const int64_t tm = (static_cast<int64_t>(p.M) + GT - 1) / GT, tn = (static_cast<int64_t>(p.N) + GT - 1) / GT;
    if (tm * tn > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(fp8_general_kernel, dim3(static_cast<unsigned>(tm * tn)), dim3(256), 0, stream, p, static_cast<int>(tn));
}

}  // namespace kda
