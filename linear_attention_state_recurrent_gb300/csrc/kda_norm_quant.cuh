// kda_norm_quant: residual addition, RMS norm and quantisation to e4m3 with a scale per row
// and group of 128 columns, in one pass over memory.
//
// A row stays in the registers of its threads between the sum of squares and the
// quantisation, so each input is read once and each output written once; the kernel is bound
// by HBM (33494 x 4096 bf16 with a residual: 142-143 us, the measured copy's rate; quantisation of
// 16480 x 4096 alone 32.5 us, 94% of it). Eight consecutive columns per thread and chunk (16 bytes of a 16-bit type) make 16
// lanes one group of 128, whose maximum is four shuffles.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_launch.h"
#include "kda_layer.h"
#include "kda_pdl.cuh"

namespace kda {
namespace {

struct Bf16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw v) { return bf16_to_f32(v); }
    static __device__ __forceinline__ raw store(float f) { return f32_to_bf16(f); }
    static __device__ __forceinline__ float2 load2(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t store2(float a, float b) { return pack_bf16x2(a, b); }
};
struct Fp16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ raw store(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ float2 load2(uint32_t u)
    {
        return make_float2(load(static_cast<uint16_t>(u)), load(static_cast<uint16_t>(u >> 16)));
    }
    static __device__ __forceinline__ uint32_t store2(float a, float b)
    {
        return static_cast<uint32_t>(store(a)) | static_cast<uint32_t>(store(b)) << 16;
    }
};
struct Fp32 {
    using raw = float;
    static __device__ __forceinline__ float load(raw v) { return v; }
    static __device__ __forceinline__ raw store(float f) { return f; }
};

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / x to within one step, for 2^-126 <= x (infinity gives 0, a NaN itself)
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// two fp32 -> two e4m3 (lo in the low byte), round to nearest even, saturating at 448; NaN stays NaN
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The E columns of a thread's chunk: contiguous (VEC: moved in 16-byte vectors, the chunk
// that the row's end cuts element by element) or 32 apart (one column per lane, so that a
// warp's scalar accesses stay coalesced). Raw holds them as they are in memory, so that the
// next row's can be on their way in few registers.
template <typename T, bool VEC, int E>
struct Raw {
    using raw = typename T::raw;
    static constexpr int VECS = E * sizeof(raw) / 16;
    union {
        uint4 v[VEC ? VECS : 1];
        raw e[E];
    };
    __device__ __forceinline__ void load(const raw *row, int c0, int D)
    {
        if (VEC && c0 + E <= D) {
#pragma unroll
            for (int i = 0; i < VECS; i++) v[i] = reinterpret_cast<const uint4 *>(row + c0)[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < E; i++) {
            const int c = c0 + (VEC ? i : 32 * i);
            e[i] = c < D ? row[c] : raw(0);
        }
    }
    __device__ __forceinline__ void get(float (&f)[E]) const
    {
        if constexpr (VEC && sizeof(raw) == 2) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 x = T::load2(w[i]);
                f[2 * i] = x.x;
                f[2 * i + 1] = x.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) f[i] = T::load(e[i]);
        }
    }
};

template <typename T, bool VEC, int E>
__device__ __forceinline__ void store_chunk(typename T::raw *row, int c0, int D, const float (&v)[E])
{
    if (VEC && c0 + E <= D) {
        if constexpr (sizeof(typename T::raw) == 2) {
            *reinterpret_cast<uint4 *>(row + c0) = make_uint4(T::store2(v[0], v[1]), T::store2(v[2], v[3]),
                                                              T::store2(v[4], v[5]), T::store2(v[6], v[7]));
        } else {
#pragma unroll
            for (int i = 0; i < E / 4; i++)
                *reinterpret_cast<float4 *>(row + c0 + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < E; i++) {
        const int c = c0 + (VEC ? i : 32 * i);
        if (c < D) row[c] = T::store(v[i]);
    }
}

constexpr float kE4m3Max = 448.f;

// TPR threads per row, CH chunks per thread; a CTA holds ROWS = max(1, 128 / TPR) rows and goes
// on to the rows a whole grid further, whose loads it has issued before it works on this one's
// values: HBM always has requests whatever the row's chain of reduction, division and stores
// takes. RES and NORM leave out the registers (and so the warps) that steps which are
// not asked for would cost.
template <typename T, bool VEC, int TPR, int CH, bool RES, bool NORM>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, VEC && sizeof(typename T::raw) == 2 && CH <= 2 ? (RES ? 1024 : 1536) / (TPR < 128 ? 128 : TPR) : 1)
norm_quant_kernel(const NormQuantParams p)
{
    constexpr int E = VEC ? 8 : 4;           // columns per chunk
    constexpr int LANES = VEC ? 16 : 32;     // lanes that hold one group of 128
    constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
    using raw = typename T::raw;
    const int t = threadIdx.x % TPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR;
    pdl_wait_then_release();

    const int D = p.D;
    auto col0 = [&](int i) {
        const int c = i * TPR + t;
        return VEC ? c * 8 : (c / 32) * 128 + (c % 32);
    };
    Raw<T, VEC, E> x[CH], res[RES ? CH : 1];
    auto fetch = [&](int64_t row) {
        const raw *px = static_cast<const raw *>(p.x) + row * p.ld_x;
#pragma unroll
        for (int i = 0; i < CH; i++) x[i].load(px, col0(i), D);
        if (RES) {
            const raw *pr = static_cast<const raw *>(p.res) + row * p.ld_res;
#pragma unroll
            for (int i = 0; i < CH; i++) res[i].load(pr, col0(i), D);
        }
    };
    if (r < p.N) fetch(r);
    // A CTA's teams of less than a warpgroup are whole warps and meet at no barrier; larger teams
    // are the CTA, whose threads all have the same row.
    for (int parity = 0; r < p.N; r += step, parity ^= 1) {
        float h[CH][E];
#pragma unroll
        for (int i = 0; i < CH; i++) {
            x[i].get(h[i]);
            if (RES) {
                float v[E];
                res[i].get(v);
#pragma unroll
                for (int j = 0; j < E; j++) h[i][j] += v[j];
            }
        }
        if (r + step < p.N) fetch(r + step);
        if (RES) {
            raw *ro = static_cast<raw *>(p.res_out) + r * p.ld_ro;
#pragma unroll
            for (int i = 0; i < CH; i++) store_chunk<T, VEC, E>(ro, col0(i), D, h[i]);
        }
        if (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < CH; i++)
#pragma unroll
                for (int j = 0; j < E; j++) ss = fmaf(h[i][j], h[i][j], ss);
            ss = warp_sum(ss);
            if (TPR > 32) {
                __shared__ float part[2][TPR / 32 > 0 ? TPR / 32 : 1];   // two rows' in turn: one barrier per row
                if (threadIdx.x % 32 == 0) part[parity][threadIdx.x / 32] = ss;
                __syncthreads();
                ss = 0.f;
#pragma unroll
                for (int i = 0; i < TPR / 32; i++) ss += part[parity][i];
            }
            const float rstd = rsqrtf(ss / static_cast<float>(D) + p.eps);
#pragma unroll
            for (int i = 0; i < CH; i++) {
                Raw<Fp32, VEC, E> w;
                w.load(p.w, col0(i), D);
#pragma unroll
                for (int j = 0; j < E; j++) h[i][j] = h[i][j] * rstd * w.e[j];
            }
        }
        if (p.y) {
            raw *y = static_cast<raw *>(p.y) + r * p.ld_y;
#pragma unroll
            for (int i = 0; i < CH; i++) store_chunk<T, VEC, E>(y, col0(i), D, h[i]);
        }
        uint8_t *q = p.q + r * p.ld_q;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < E; j++) m = max_nan(m, fabsf(h[i][j]));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            // A product with 1 / 448 in place of a division: the scale is off by at most 2^-23.
            const float s = max_nan(m, kE4m3Max * 1.17549435e-38f) * (1.f / kE4m3Max);
            // y / s as fp32 rounds it, so that q is its nearest even also where it lies between two values of e4m3: the
            // product with the reciprocal and what it leaves over, taken to the quotient (Markstein 1990), two columns at a time (16480 x 4096
            // alone: 32.5 us, one at a time 34.5, without the remainder 31.8 but one exact midpoint in ten rounded to odd).
            const float inv = reciprocal(s), less = s < INFINITY ? -s : 0.f;
            auto quotients = [&](float a, float b) {
                const float2 y = make_float2(a, b), c = make_float2(inv, inv), t = fmul2(y, c);
                const float2 v = ffma2(ffma2(t, make_float2(less, less), y), c, t);
                return pack_e4m3x2(v.x, v.y);
            };
            const int c0 = col0(i);
            if (c0 < D) {
                if (t % LANES == 0) p.s[r * p.s_row + static_cast<int64_t>(c0 / 128) * p.s_group] = s;
                if (VEC && c0 + E <= D) {
                    const uint32_t lo = quotients(h[i][0], h[i][1]) | static_cast<uint32_t>(quotients(h[i][2], h[i][3])) << 16;
                    const uint32_t hi = quotients(h[i][E - 4], h[i][E - 3]) | static_cast<uint32_t>(quotients(h[i][E - 2], h[i][E - 1])) << 16;
                    *reinterpret_cast<uint2 *>(q + c0) = make_uint2(lo, hi);
                } else {
#pragma unroll
                    for (int j = 0; j < E; j += 2) {
                        const int c = c0 + (VEC ? j : 32 * j), next = c + (VEC ? 1 : 32);
                        const uint16_t two = quotients(h[i][j], h[i][j + 1]);
                        if (c < D) q[c] = static_cast<uint8_t>(two);
                        if (next < D) q[next] = static_cast<uint8_t>(two >> 8);
                    }
                }
            }
            __syncwarp();
        }
    }
}

// One launch over as many CTAs as run at once.
template <typename T, bool VEC, int TPR, int CH, bool RES, bool NORM>
cudaError_t go(const NormQuantParams &p, cudaStream_t stream)
{
    constexpr int rows = TPR < 128 ? 128 / TPR : 1, threads = TPR < 128 ? 128 : TPR;
    const auto kernel = norm_quant_kernel<T, VEC, TPR, CH, RES, NORM>;
    static std::atomic<int> known[64];   // per device, once a query has answered
    int dev = 0, resident = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev < 64;
    if (kept) resident = known[dev].load(std::memory_order_relaxed);
    if (resident == 0) {
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, 0)) != cudaSuccess)
            return e;
        resident *= sms;
        if (resident < 1) return cudaErrorInvalidConfiguration;
        if (kept) known[dev].store(resident, std::memory_order_relaxed);
    }
    const int64_t want = (p.N + rows - 1) / rows;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(want < resident ? want : resident)), dim3(threads), 0, stream, p);
}

template <typename T, bool VEC, int TPR, int CH>
cudaError_t run(const NormQuantParams &p, cudaStream_t stream)
{
    if (p.res) return p.w ? go<T, VEC, TPR, CH, true, true>(p, stream) : go<T, VEC, TPR, CH, true, false>(p, stream);
    return p.w ? go<T, VEC, TPR, CH, false, true>(p, stream) : go<T, VEC, TPR, CH, false, false>(p, stream);
}

// The smallest team that holds a row with two chunks per thread where there are rows enough to
// fill the GPU (more chunks cost the warps that hide the loads), one per thread (more threads, a
// shorter chain) where there are not.
template <typename T>
cudaError_t pick_vectors(const NormQuantParams &p, cudaStream_t stream)
{
    const int chunks = (p.D + 7) / 8;
    const bool many = p.N >= 512;
    if (chunks <= 32) return run<T, true, 32, 1>(p, stream);
    if (many && chunks <= 64) return run<T, true, 32, 2>(p, stream);
    if (chunks <= 128) return run<T, true, 128, 1>(p, stream);
    if (many && chunks <= 256) return run<T, true, 128, 2>(p, stream);
    if (many && chunks <= 512) return run<T, true, 256, 2>(p, stream);
    if (chunks <= 512) return run<T, true, 512, 1>(p, stream);
    if (chunks <= 1024) return run<T, true, 512, 2>(p, stream);
    if (chunks <= 1536) return run<T, true, 512, 3>(p, stream);
    if constexpr (sizeof(typename T::raw) == 2)
        if (chunks <= 2048) return run<T, true, 1024, 2>(p, stream);
    if (chunks <= 2048) return run<T, true, 512, 4>(p, stream);
    return run<T, true, 512, 8>(p, stream);
}

// Single elements: four columns per chunk and little in flight per register, so more chunks per
// thread, in teams that leave few threads without a column (20000 x 2051 bf16: 120 us in 256 threads
// of three chunks, 151 in 512 of two).
template <typename T>
cudaError_t pick_elements(const NormQuantParams &p, cudaStream_t stream)
{
    const int chunks = (p.D + 127) / 128 * 32;
    const bool many = p.N >= 512;
    if (chunks <= 32) return run<T, false, 32, 1>(p, stream);
    if (many && chunks <= 128) return run<T, false, 32, 4>(p, stream);
    if (chunks <= 128) return run<T, false, 128, 1>(p, stream);
    if (many && chunks <= 256) return run<T, false, 128, 2>(p, stream);
    if (many && chunks <= 384) return run<T, false, 128, 3>(p, stream);
    if (many && chunks <= 512) return run<T, false, 128, 4>(p, stream);
    if (chunks <= 512) return run<T, false, 512, 1>(p, stream);
    if (chunks <= 768) return run<T, false, 256, 3>(p, stream);
    if (chunks <= 1024) return run<T, false, 256, 4>(p, stream);
    if (chunks <= 1536) return run<T, false, 512, 3>(p, stream);
    if (chunks <= 2048) return run<T, false, 512, 4>(p, stream);
    if (chunks <= 2560) return run<T, false, 512, 5>(p, stream);
    if (chunks <= 4096) return run<T, false, 512, 8>(p, stream);
    return run<T, false, 512, 16>(p, stream);
}

template <typename T>
cudaError_t by_alignment(const NormQuantParams &p, cudaStream_t stream)
{
    const size_t es = sizeof(typename T::raw);
    auto ok = [&](const void *b, int64_t ld) {
        return !b || (reinterpret_cast<uintptr_t>(b) % 16 == 0 && ld * es % 16 == 0);
    };
    const bool vec = ok(p.x, p.ld_x) && ok(p.res, p.ld_res) && ok(p.res_out, p.ld_ro) && ok(p.y, p.ld_y) &&
                     reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && p.ld_q % 8 == 0;
    return vec ? pick_vectors<T>(p, stream) : pick_elements<T>(p, stream);
}

}  // namespace
}  // namespace kda
