// Device helpers of the gated delta rule's kernels: slots, lengths, the scalar gate, and the two-term bf16 and tf32
// forms in which fp32 values enter the tensor cores.
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
__device__ __forceinline__ float log_decay(uint16_t raw_g, float expA, float dtb) { return bounded(-expA * softplus_f(bf16_to_f32(raw_g) + dtb)); }

// x and y as packed bf16 pairs hi + lo: hi is x rounded to bf16 and lo what is left, rounded again, so that
// |x - hi - lo| <= 2^-17 |x|.
__device__ __forceinline__ float2 left(float2 x, uint32_t hi)
{
    return fsub2(x, make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
}
__device__ __forceinline__ uint32_t rest2(float x, float y, uint32_t hi)
{
    const float2 d = left(make_float2(x, y), hi);
    return pack_bf16x2(d.x, d.y);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x, y);
    lo = rest2(x, y, hi);
}

// fp32 values as two tf32 terms, truncated: |x - hi - lo| <= 2^-20 |x|. (Not volatile: the order of products of different sums is free,
// 61 x 5 rows x 12 heads 14.2 us for 14.7.)
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <int N>
struct Tf32 {
    uint32_t hi[N], lo[N];
    __device__ __forceinline__ void set(int i, float x)
    {
        hi[i] = __float_as_uint(x) & 0xffffe000u;
        lo[i] = __float_as_uint(x - __uint_as_float(hi[i]));
    }
};
__device__ __forceinline__ void mma_split(float (&d)[4], const Tf32<4> &a, const Tf32<2> &b)
{
    mma_tf32(d, a.lo, b.hi);
    mma_tf32(d, a.hi, b.lo);
    mma_tf32(d, a.hi, b.hi);
}

// Sums of log-decays. What is needed are their differences, to an absolute error of 2^-24: a few tokens with little decay may follow
// thousands of nats. So they are taken in integers, hi 2^-8 + lo 2^-32 (each term off by 2^-33; bounded at 1000 in magnitude, 64 of them
// keep hi below 2^24 and lo below 2^30), and kept as two floats. (In 64-bit floats, of which a multiprocessor adds two
// a clock, 16 requests of 8 rows x 32 heads took 18.9 us for 18.4.)
struct FixedDecay {
    int hi, lo;
    __device__ __forceinline__ static FixedDecay of(float g)
    {
        const float h = rintf(g * 256.f);
        return {static_cast<int>(h), __float2int_rn((g - h * 0.00390625f) * 4294967296.f)};
    }
    __device__ __forceinline__ FixedDecay operator+(const FixedDecay &o) const { return {hi + o.hi, lo + o.lo}; }
    // the two floats; `nan`: one of the terms was
    __device__ __forceinline__ float2 get(bool nan) const
    {
        return make_float2(nan ? __int_as_float(0x7fffffff) : static_cast<float>(hi) * 0.00390625f, static_cast<float>(lo) * 2.3283064365386963e-10f);
    }
    // of lanes 0 .. own
    __device__ __forceinline__ FixedDecay up_to(int lanes) const
    {
        FixedDecay s = *this;
        for (int o = 1; o < lanes; o <<= 1) {
            const int h = __shfl_up_sync(0xffffffffu, s.hi, o), l = __shfl_up_sync(0xffffffffu, s.lo, o);
            if (static_cast<int>(threadIdx.x & 31) >= o) s = s + FixedDecay{h, l};
        }
        return s;
    }
};
// Whether a lane below the own one says so.
__device__ __forceinline__ bool any_below(bool x) { return (__ballot_sync(0xffffffffu, x) & ((1u << (threadIdx.x & 31)) - 1)) != 0; }

// The sum of a warp's log-decays up to each lane.
struct RunningDecay {
    struct At {
        float hi, lo;
        __device__ __forceinline__ float operator-(const At &o) const { return (hi - o.hi) + (lo - o.lo); }
        __device__ __forceinline__ operator float() const { return hi + lo; }
    };
    At own;
    __device__ __forceinline__ RunningDecay(float g, int lanes)
    {
        const float2 x = FixedDecay::of(g).up_to(lanes).get(any_below(g != g) || g != g);
        own = {x.x, x.y};
    }
    __device__ __forceinline__ At of(int lane) const
    {
        return {__shfl_sync(0xffffffffu, own.hi, lane), __shfl_sync(0xffffffffu, own.lo, lane)};
    }
};

}  // namespace gdn
}  // namespace kda
