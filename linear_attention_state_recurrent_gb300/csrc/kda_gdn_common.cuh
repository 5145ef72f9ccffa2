// Device helpers of the gated delta rule's kernels: slots, lengths, the scalar gate, and the two-term bf16 form in
// which fp32 values enter the tensor cores.
#pragma once

#include "kda_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_gdn.h"

namespace kda {
namespace gdn {

constexpr uint32_t kErrLengths = 16u;   // KDA_ERRFLAG_LENGTHS

// (Not a read-only load: the compiler may take one ahead of the wait for the kernel that writes the indices. So too with
// lengths, and with what one of a call's kernels leaves to the next.)
__device__ __forceinline__ int64_t load_slot(const GdnParams &p, int64_t e) { return static_cast<int64_t>(p.indices[e * p.index_stride]); }

// A log-decay that differences of sums are taken of: below -1000 e^x and 2^x are 0 in fp32, and sums of what is below it
// (-inf, for a large A_log or raw_g) have no differences. NaN stays NaN.
__device__ __forceinline__ float bounded(float g) { return g < -1000.f ? -1000.f : g; }

// Log-decay of a token and head: -e^{A_log} softplus(raw_g + dt_bias).
__device__ __forceinline__ float log_decay(const GdnParams &p, int64_t row, int h, float expA, float dtb)
{
    return bounded(-expA * softplus_f(bf16_to_f32(p.rg[row * p.ld_g + h]) + dtb));
}

// x and y as packed bf16 pairs hi + lo: hi is x rounded to bf16 and lo what is left, rounded again, so that
// |x - hi - lo| <= 2^-17 |x|.
__device__ __forceinline__ uint32_t rest2(float x, float y, uint32_t hi)
{
    const float2 d = fsub2(make_float2(x, y), make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
    return pack_bf16x2(d.x, d.y);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x, y);
    lo = rest2(x, y, hi);
}

// The sum of a warp's log-decays up to each lane. What is needed are differences of such sums, to an absolute error of
// 2^-24: a few tokens with little decay may follow thousands of nats. So the sums are taken in 64 bits and kept as two floats.
struct RunningDecay {
    struct At {
        float hi, lo;
        __device__ __forceinline__ float operator-(const At &o) const { return (hi - o.hi) + (lo - o.lo); }
    };
    At own;
    __device__ __forceinline__ RunningDecay(float g, int lanes)
    {
        double b = g;
        for (int o = 1; o < lanes; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, b, o);
            if (static_cast<int>(threadIdx.x & 31) >= o) b += x;
        }
        own.hi = static_cast<float>(b);
        own.lo = static_cast<float>(b - own.hi);
    }
    __device__ __forceinline__ At of(int lane) const
    {
        return {__shfl_sync(0xffffffffu, own.hi, lane), __shfl_sync(0xffffffffu, own.lo, lane)};
    }
};

}  // namespace gdn
}  // namespace kda
