// kda_fp8_matmul: out = A W^T with e4m3 operands and a scale for each block of 128.
//
//   out[m, n] = sum_g sa[m, g] sw[n / 128, g] * (sum_{k in g} a[m, k] w[n, k])
//
// The inner sums of one group g (128 k: four tcgen05.mma steps of 32) go to a fresh
// accumulator in tensor memory; as the tensor core forms the next group in another buffer,
// the epilogue warps read the finished one, scale it and add it to sums they hold in fp32
// registers. TMA brings 128-byte-wide tiles (one group) with the 128-byte swizzle that the
// matrix descriptors name; columns past K and rows past the matrix read as zeros.
//
// Three arrangements (times on a GB300 for K = 4096; `wide` writes bf16):
//  - thin_kernel, up to 64 rows of A: 128 rows of W are the MMA's M side, the rows of A its N side.
//    Bound by the stream of weights: M = 1, N = 20512 17.1-17.4 us = 4.9 TB/s, of which the stream alone
//    (no MMA, no epilogue) is 15.6 us, and a plain kernel that reads as many bytes 16.9 us; N = 4096 5.2 us.
//  - slim_kernel, up to 128 rows of A per CTA and a tile of W that makes the CTAs fill the GPU once:
//    M = 128, N = 20512 21.0-21.4 us. The stream alone is 15.1 us, with the MMAs 18.6, the rest the sums; that each CTA
//    copies all rows of A again costs nothing (kept in shared memory from the first turn on: the same times).
//    In both the inner axis may be split over a cluster whose CTAs join their sums through distributed
//    shared memory in a fixed order.
//  - wide_kernel: tiles of 256 x 256 by a pair of CTAs (cta_group::2), persistent: M = 33494,
//    N = 20512 2.19-2.28 ms = 2.47-2.57 PFLOP/s (the card's clock falls under it), 59% of the tensor pipe's cycles.
//    Of the 490 ns a group takes, the copies alone need 225 and the MMAs alone 287; MMAs and copies with every
//    accumulator handed back unread take 359, read but not added up 427, and all of it without copies 447. So it
//    is the way of an accumulator through the epilogue and back that bounds it, with the two that tensor memory holds.
//    Measured and not kept: four accumulators of 128 columns (2.46 ms against 2.22),
//    tiles of 192 with one load per group (2.36), loads of tensor memory overlapped across groups
//    (2.49), the MMA loop unrolled over the ring (2.42, registers), one polling warp of four (2.35).
// Operands that TMA cannot address (rows off 16-byte boundaries) take general_kernel, on the FMA units: 1000 x 4096 x
// 4095 1.97 ms, where rows padded to 16 bytes take 20 us.
#include <atomic>
#include <climits>
#include <cstdint>
#include <mutex>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "kda_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_launch.h"
#include "kda_layer.h"
#include "kda_pdl.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

// ---- pieces shared by the tensor-core kernels ---------------------------------------------

// Matrix descriptor of a K-major tile of 128-byte rows with the 128-byte swizzle: groups of 8
// rows follow each other at 1024 bytes; the tile starts on a 1024-byte boundary. One MMA step
// of 32 k is 32 bytes further. `at16`: shared-memory address / 16.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t at16)
{
    constexpr uint32_t HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
    return static_cast<uint64_t>(HIGH) << 32 | (1u << 16) | at16;
}

// D (+)= A B^T of 32 k, e4m3 operands (format 0 of kind::f8f6f4), fp32 sums.
template <int CG, bool ADD>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc)
{
    if (CG == 1)
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                     " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0));
    else
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                     " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0));
}

// D = A B^T of one group of 128 k.
template <int CG>
__device__ __forceinline__ void mma_group(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    const uint32_t a16 = a >> 4, b16 = b >> 4;
    mma_step<CG, false>(d, desc_sw128(a16), desc_sw128(b16), idesc);
#pragma unroll
    for (int s = 1; s < 4; s++) mma_step<CG, true>(d, desc_sw128(a16 + 2 * s), desc_sw128(b16 + 2 * s), idesc);
}

// Waits for the mbarrier phase with the given parity; gives up after 4e9 clocks (~2 s). The
// clock is read only every 64 tries: a wait here is on the path from one group to the next.
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity)
{
    long long start = 0;
    for (uint32_t it = 1;; it++) {
        uint32_t ok;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(mbar), "r"(parity) : "memory");
        if (ok) return true;
        if (it % 64 == 0) {
            const long long now = clock64();
            if (it == 64) start = now;
            else if (now - start > 4000000000ll) return false;
        }
    }
}

// The same by a converged warp, with one answer for all its lanes: what follows is instructions of the whole warp.
__device__ __forceinline__ bool wait_warp(uint32_t mbar, uint32_t parity)
{
    return __all_sync(0xffffffffu, wait_phase(mbar, parity));
}

// An arrival on the barrier at this place in both CTAs of the pair once its MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(mbar), "h"(static_cast<uint16_t>(3)) : "memory");
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}

// Whether the phase with the given parity is over, without waiting.
__device__ __forceinline__ bool test_phase(uint32_t mbar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(mbar), "r"(parity) : "memory");
    return ok;
}

// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();   // warps come here from loops that each lane left for itself
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address in CTA `rank` of the cluster of a shared-memory address of this CTA
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Whether a CTA of the cluster has said, in the word at `failed` of its own shared memory, that it lacks sums of a
// split's. By a whole warp, each lane asking one CTA.
__device__ __forceinline__ bool any_failed(uint32_t failed, int split)
{
    const uint32_t k = threadIdx.x % 32;
    uint32_t v = 0;
    if (k < static_cast<uint32_t>(split)) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cta(failed, k)));
    return __any_sync(0xffffffffu, v != 0);
}
// Arrival on a barrier of any CTA of the cluster. What it orders are the reads of tensor memory,
// by the tcgen05 fence in front of it; a release at cluster scope would wait for every
// access of the thread each time (a third of the kernel's time, measured).
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void arrive_local(uint32_t mbar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(mbar) : "memory");
}
// 4-byte asynchronous global -> shared copy
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void store_out(void *out, int64_t i, int dtype, float v)
{
    if (dtype == 0) static_cast<uint16_t *>(out)[i] = f32_to_bf16(v);
    else if (dtype == 1) static_cast<__half *>(out)[i] = __float2half_rn(v);
    else static_cast<float *>(out)[i] = v;
}

__device__ __forceinline__ void report(const Fp8Params &p)
{
    if (p.err) atomicOr(p.err, kErrTimeout);
}

// The end of a role, also of one that has given up: no CTA ends, and no ring takes sums, with copies or MMAs of its
// own in flight. Nothing is waited for here that the roles after it in the chain have not waited for, if all went well.
// Copies: the last turn of stages 0 .. n - 1 (barriers from `full` on), where the next load would have been stage s in
// the turn of parity `phase`.
__device__ __forceinline__ void landed(uint32_t full, int n, int s, uint32_t phase, const Fp8Params &p)
{
    for (int i = 0; i < n; i++)
        if (!wait_phase(full + i * 8, i < s ? phase ^ 1u : phase)) { report(p); break; }
}
// MMAs: the last commits, on the ring's stage before `s` and on the accumulator before `b` of the turns of parity
// `phase` and `tphase` (the MMA warp's own, as it left its loop).
__device__ __forceinline__ void finished(uint32_t empty, int stages, int s, uint32_t phase, uint32_t tfull, int nbuf, int b,
                                         uint32_t tphase, const Fp8Params &p)
{
    if (!wait_warp(empty + (s > 0 ? s - 1 : stages - 1) * 8, s > 0 ? phase : phase ^ 1u) ||
        !wait_warp(tfull + (b > 0 ? b - 1 : nbuf - 1) * 8, b > 0 ? tphase ^ 1u : tphase))
        report(p);
}

constexpr int BK = 128;                       // bytes (= k) per group

// ---- a handful of rows of A ---------------------------------------------------------------

// 128 rows of W are the MMA's M side and NT rows of A its N side, so that all four quarters of
// the TMEM lanes have work and an epilogue thread holds only NT (or NT / 2) sums: its time per
// group is what the stream of weights would otherwise wait for.
template <int NT>
struct Thin {
    static constexpr int EW = NT > 32 ? 8 : 4;              // epilogue warps
    static constexpr int THREADS = 128 + EW * 32;           // copies, MMAs, scales, one idle warp, then the epilogue's
    static constexpr int COLS = NT * 4 / EW;                // columns (rows of A) per epilogue thread
    static constexpr int NBUF = 4;                          // accumulators in tensor memory
    static constexpr int STAGE = 128 * BK + NT * BK;
    static constexpr int STAGES = NT > 32 ? 4 : NT > 16 ? 5 : 6;
    static constexpr int SR = 8, SLOT = NT + 4;             // groups of scales in flight: NT rows' and the tile's of W
    static constexpr int SMEM = 1024 + STAGES * STAGE;      // two CTAs per SM
};

template <int NT>
__global__ void __launch_bounds__(Thin<NT>::THREADS, 2)
thin_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const Fp8Params p,
            const int split)
{
    using C = Thin<NT>;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ uint64_t bars[2 * C::STAGES + 2 * C::NBUF + 2 * C::SR];
    __shared__ uint32_t tmem_base, failed;
    __shared__ alignas(16) float scales[C::SR][C::SLOT];
    const uint32_t ring = (tc::smem_addr(dyn) + 1023u) & ~1023u;
    float *red = reinterpret_cast<float *>(dyn + (ring - tc::smem_addr(dyn)));   // the ring again, once it is drained
    const uint32_t b0 = tc::smem_addr(bars);
    auto full = [&](int s) { return b0 + s * 8; };
    auto empty = [&](int s) { return b0 + (C::STAGES + s) * 8; };
    auto tfull = [&](int b) { return b0 + (2 * C::STAGES + b) * 8; };
    auto tempty = [&](int b) { return b0 + (2 * C::STAGES + C::NBUF + b) * 8; };
    auto sfull = [&](int r) { return b0 + (2 * C::STAGES + 2 * C::NBUF + r) * 8; };
    auto sempty = [&](int r) { return b0 + (2 * C::STAGES + 2 * C::NBUF + C::SR + r) * 8; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % split;
    const int n0 = blockIdx.x / split * 128, t0 = blockIdx.y * NT;
    const int groups = (p.K + BK - 1) / BK;
    const int g0 = static_cast<int>(static_cast<int64_t>(groups) * rank / split);
    const int g1 = static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / split);
    auto load = [&](int g, int s) {
        const uint32_t at = ring + s * C::STAGE;
        tc::mbar_expect_tx(full(s), C::STAGE);
        tc::tma_load_2d(at, &tm_w, g * BK, n0, full(s));
        tc::tma_load_2d(at + 128 * BK, &tm_a, g * BK, t0, full(s));
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; s++) { tc::mbar_init(full(s), 1); tc::mbar_init(empty(s), 1); }
        for (int b = 0; b < C::NBUF; b++) { tc::mbar_init(tfull(b), 1); tc::mbar_init(tempty(b), C::EW); }
        for (int r = 0; r < C::SR; r++) { tc::mbar_init(sfull(r), 32); tc::mbar_init(sempty(r), C::EW); }
        failed = 0;
        tc::prefetch_tensormap(&tm_w);
        tc::prefetch_tensormap(&tm_a);
    }
    pdl_wait();
    // the ring's first turn needs nothing but its barriers, which this thread has made
    const int ahead = min(C::STAGES, g1 - g0);
    if (threadIdx.x == 0)
        for (int i = 0; i < ahead; i++) load(g0 + i, i);
    // tensor memory is taken before the next grid may start: it could hold what this one waits for
    if (warp == 1) tc::tmem_alloc<C::NBUF * NT>(tc::smem_addr(&tmem_base));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_release();

    const uint32_t tmem = tmem_base;
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            for (int g = g0 + ahead; g < g1; g++) {
                if (!wait_phase(empty(s), phase)) { report(p); break; }
                load(g, s);
                if (++s == C::STAGES) { s = 0; phase ^= 1; }
            }
            landed(full(0), ahead, s, phase, p);
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t ID = tc::instr_desc(0, 128, NT);
        int s = 0, b = 0, r = 0;
        uint32_t phase = 0, tphase = 1, sphase = 0;
        bool ok = true;
        for (int g = g0; g < g1; g++) {
            // the scales too, for the epilogue, which then waits for the products alone
            if (!wait_phase(full(s), phase) || !wait_phase(sfull(r), sphase) || !wait_phase(tempty(b), tphase)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) { report(p); break; }
            tc::fence_after_sync();
            const uint32_t at = ring + s * C::STAGE;
            if (elect_one()) {
                mma_group<1>(tmem + b * NT, at, at + 128 * BK, ID);
                tc::commit(empty(s));
                tc::commit(tfull(b));
            }
            __syncwarp();
            if (++s == C::STAGES) { s = 0; phase ^= 1; }
            if (++b == C::NBUF) { b = 0; tphase ^= 1; }
            if (++r == C::SR) { r = 0; sphase ^= 1; }
        }
        finished(empty(0), C::STAGES, s, phase, tfull(0), C::NBUF, b, tphase, p);
    } else if (warp == 2 && rank != p.stalled) {
        int r = 0;
        uint32_t phase = 1;
        const float *sa = p.sa + (t0 + lane) * p.sa_row + g0 * p.sa_group;
        const float *sw = p.sw + static_cast<int64_t>(n0 / 128) * p.sw_row + g0 * p.sw_group;
        for (int g = g0; g < g1; g++) {
            if (!wait_phase(sempty(r), phase)) { report(p); break; }
            const uint32_t at = tc::smem_addr(&scales[r][0]);
#pragma unroll
            for (int j = 0; j < NT; j += 32)
                if (lane + j < NT && t0 + lane + j < p.M) cp_async4(at + (lane + j) * 4, sa + j * p.sa_row);
            if (lane == 0) cp_async4(at + NT * 4, sw);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(sfull(r)) : "memory");
            sa += p.sa_group;
            sw += p.sw_group;
            if (++r == C::SR) { r = 0; phase ^= 1; }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        const int quarter = warp % 4, c0 = (warp - 4) / 4 * C::COLS;
        const int n = quarter * 32 + lane;                    // row of W within the tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c0;
        float acc[C::COLS];
#pragma unroll
        for (int c = 0; c < C::COLS; c++) acc[c] = 0.f;
        int b = 0, r = 0;
        uint32_t tphase = 0;
        bool ok = true;
        for (int g = g0; g < g1; g++) {
            if (!wait_warp(tfull(b), tphase)) { ok = false; break; }
            tc::fence_after_sync();
            float v[C::COLS / 16][16];
#pragma unroll
            for (int c = 0; c < C::COLS / 16; c++) tc::tmem_ld16(lanes + b * NT + c * 16, v[c]);
            const float4 *f4 = reinterpret_cast<const float4 *>(&scales[r][c0]);
            const float sw = scales[r][NT];
            tc::tmem_ld_wait();
            tc::fence_before_sync();
            if (lane == 0) arrive_local(tempty(b));
#pragma unroll
            for (int c = 0; c < C::COLS / 4; c++) {
                const float4 f = f4[c];
                acc[4 * c] = fmaf(v[c / 4][4 * (c % 4)], f.x * sw, acc[4 * c]);
                acc[4 * c + 1] = fmaf(v[c / 4][4 * (c % 4) + 1], f.y * sw, acc[4 * c + 1]);
                acc[4 * c + 2] = fmaf(v[c / 4][4 * (c % 4) + 2], f.z * sw, acc[4 * c + 2]);
                acc[4 * c + 3] = fmaf(v[c / 4][4 * (c % 4) + 3], f.w * sw, acc[4 * c + 3]);
            }
            __syncwarp();
            if (lane == 0) arrive_local(sempty(r));
            if (++b == C::NBUF) { b = 0; tphase ^= 1; }
            if (++r == C::SR) r = 0;
        }
        if (!ok) {
            report(p);
            failed = 1;   // the ring may still be written and read; what this warp was to store stays as it was
        } else if (split > 1) {
#pragma unroll
            for (int c = 0; c < C::COLS; c++) red[(c0 + c) * 128 + n] = acc[c];
        } else if (n0 + n < p.N) {
#pragma unroll
            for (int c = 0; c < C::COLS; c++)
                if (t0 + c0 + c < p.M)
                    store_out(p.out, static_cast<int64_t>(t0 + c0 + c) * p.ld_out + n0 + n, p.out_dtype, acc[c]);
        }
    }
    if (split > 1) {
        cluster_sync();
        if (warp >= 4 && !any_failed(tc::smem_addr(&failed), split)) {
            // CTA `rank` joins the rows rank, rank + split, ... of A, over the CTAs in order
            const int e = threadIdx.x - 128, n = e % 128;
            const int rows = min(NT, p.M - t0);
            uint32_t part[8];
#pragma unroll
            for (int k = 0; k < 8; k++) part[k] = in_cta(ring, k < split ? k : 0);
#pragma unroll 4
            for (int t = rank + (e / 128) * split; t < rows; t += split * (C::EW / 4)) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    v[k] = 0.f;
                    if (k < split) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[k]) : "r"(part[k] + (t * 128 + n) * 4));
                }
                float sum = v[0];
#pragma unroll
                for (int k = 1; k < 8; k++) sum += v[k];
                if (n0 + n < p.N) store_out(p.out, static_cast<int64_t>(t0 + t) * p.ld_out + n0 + n, p.out_dtype, sum);
            }
        }
        cluster_sync();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc<C::NBUF * NT>(tmem);
}

// ---- few rows of A ------------------------------------------------------------------------

// How a call is cut up: tiles of `bn` rows of W (a multiple of 16, chosen so that the CTAs fill the
// GPU once), the inner axis over a cluster of `split` CTAs, 128 rows of A per blockIdx.y of which
// `rows` (a multiple of 8) are copied.
struct SlimPlan {
    int bn, split, rows, stages, nbuf;   // nbuf accumulators of bn TMEM columns
};

struct Slim {
    static constexpr int EW = 16;                       // epilogue warps: four strips of columns x four quarters of TMEM lanes
    static constexpr int THREADS = 128 + EW * 32;       // copies, MMAs, scales, one idle warp, then the epilogue's
    static constexpr int REGS_CONTROL = 32, REGS_EPILOGUE = 112;   // 640 * 96 at launch
    static constexpr int MAX_STAGES = 12, MAX_BUF = 4;
    static constexpr int SR = 4, SLOT = 132;            // groups of scales in flight: 128 rows' and up to three blocks' of W
    static constexpr int TAIL = SR * SLOT * 4 + (2 * MAX_STAGES + 2 * MAX_BUF + 2 * SR) * 8 + 16;
    static constexpr int RING = 227 * 1024 - TAIL, FAILED = RING + TAIL - 12;   // the word any_failed reads, from `dyn` on
};

__device__ __forceinline__ void store16(const Fp8Params &p, int64_t m, int n, const float (&v)[16])
{
    const int es = p.out_dtype == 2 ? 4 : 2;
    unsigned char *o = static_cast<unsigned char *>(p.out) + (m * p.ld_out + n) * es;
    if (n + 16 <= p.N && reinterpret_cast<uintptr_t>(o) % 16 == 0) {
        if (p.out_dtype == 2) {
#pragma unroll
            for (int j = 0; j < 4; j++)
                reinterpret_cast<float4 *>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                w[j] = p.out_dtype == 0 ? pack_bf16x2(v[2 * j], v[2 * j + 1]) : tc::pack_f16x2(v[2 * j], v[2 * j + 1]);
            reinterpret_cast<uint4 *>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4 *>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; j++)
        if (n + j < p.N) store_out(p.out, m * p.ld_out + n + j, p.out_dtype, v[j]);
}

// The join of a split's sums by the epilogue warps: CTA `rank` joins the rows rank, rank + split, ... of the tile, over
// the CTAs in order. No part of the kernel's body, where its registers were spills around the groups' loop (128 x
// 20512 x 4096, not split: 22.0 us instead of 21.5).
__device__ __noinline__ void slim_join(void *out, int64_t ld_out, int out_dtype, int cols, int bn, int split, uint32_t ring, int m0,
                                       int n0, int rows, int rank)
{
    if (any_failed(ring + Slim::FAILED, split)) return;
    const int total = (rows - rank + split - 1) / split * cols;
    uint32_t part[8];
#pragma unroll
    for (int k = 0; k < 8; k++) part[k] = in_cta(ring, k < split ? k : 0);
#pragma unroll 4
    for (int i = threadIdx.x - 128; i < total; i += Slim::EW * 32) {
        const int row = i / cols * split + rank, n = i % cols;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            v[k] = 0.f;
            if (k < split)
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[k]) : "r"(part[k] + (row * (bn + 1) + n) * 4));
        }
        float sum = v[0];
#pragma unroll
        for (int k = 1; k < 8; k++) sum += v[k];
        store_out(out, static_cast<int64_t>(m0 + row) * ld_out + n0 + n, out_dtype, sum);
    }
}

// MAXC: chunks of 16 columns that an epilogue warp holds at most
template <int MAXC>
__global__ void __launch_bounds__(Slim::THREADS, 1)
slim_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const Fp8Params p,
            const SlimPlan q)
{
    using C = Slim;
    extern __shared__ __align__(1024) unsigned char dyn[];
    const uint32_t ring = tc::smem_addr(dyn), wring = ring + q.stages * q.rows * BK;
    float *scales = reinterpret_cast<float *>(dyn + C::RING);
    const uint32_t b0 = tc::smem_addr(scales) + C::SR * C::SLOT * 4;
    volatile uint32_t *tmem_base = reinterpret_cast<uint32_t *>(dyn + C::RING + C::TAIL - 16);
    auto full = [&](int s) { return b0 + s * 8; };
    auto empty = [&](int s) { return b0 + (C::MAX_STAGES + s) * 8; };
    auto tfull = [&](int b) { return b0 + (2 * C::MAX_STAGES + b) * 8; };
    auto tempty = [&](int b) { return b0 + (2 * C::MAX_STAGES + C::MAX_BUF + b) * 8; };
    auto sfull = [&](int r) { return b0 + (2 * C::MAX_STAGES + 2 * C::MAX_BUF + r) * 8; };
    auto sempty = [&](int r) { return b0 + (2 * C::MAX_STAGES + 2 * C::MAX_BUF + C::SR + r) * 8; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % q.split;
    const int groups = (p.K + BK - 1) / BK;
    const int g0 = static_cast<int>(static_cast<int64_t>(groups) * rank / q.split);
    const int g1 = static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / q.split);
    const int n0 = blockIdx.x / q.split * q.bn, m0 = blockIdx.y * 128;
    const int rows = min(128, p.M - m0);                       // live rows of A
    const int chunks = q.bn / 16, per = (chunks + 3) / 4;      // of 16 columns, per strip
    const int working = (rows + 31) / 32 * ((chunks + per - 1) / per);   // epilogue warps with something to do
    auto load = [&](int g, int s) {
        tc::mbar_expect_tx(full(s), (q.rows + q.bn) * BK);
        tc::tma_load_2d(wring + s * q.bn * BK, &tm_w, g * BK, n0, full(s));
        tc::tma_load_2d(ring + s * q.rows * BK, &tm_a, g * BK, m0, full(s));
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; s++) { tc::mbar_init(full(s), 1); tc::mbar_init(empty(s), 1); }
        for (int b = 0; b < q.nbuf; b++) { tc::mbar_init(tfull(b), 1); tc::mbar_init(tempty(b), working); }
        for (int r = 0; r < C::SR; r++) { tc::mbar_init(sfull(r), 32); tc::mbar_init(sempty(r), working); }
        *reinterpret_cast<volatile uint32_t *>(dyn + C::FAILED) = 0;
        tc::prefetch_tensormap(&tm_w);
        tc::prefetch_tensormap(&tm_a);
    }
    pdl_wait();
    // the ring's first turn needs nothing but its barriers, which this thread has made
    const int ahead = min(q.stages, g1 - g0);
    if (threadIdx.x == 0)
        for (int i = 0; i < ahead; i++) load(g0 + i, i);
    // tensor memory is taken before the next grid may start: it could hold what this one waits for
    if (warp == 1) tc::tmem_alloc<512>(b0 + (2 * C::MAX_STAGES + 2 * C::MAX_BUF + 2 * C::SR) * 8);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_release();

    const uint32_t tmem = *tmem_base;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::REGS_CONTROL));
        if (warp == 0) {
            if (lane == 0) {
                int s = 0;
                uint32_t phase = 0;
                for (int g = g0 + ahead; g < g1; g++) {
                    if (!wait_phase(empty(s), phase)) { report(p); break; }
                    load(g, s);
                    if (++s == q.stages) { s = 0; phase ^= 1; }
                }
                landed(full(0), ahead, s, phase, p);
            }
            __syncwarp();
        } else if (warp == 1) {
            // The MMA takes 128 rows of A whatever is there: those past the `rows` copied are other
            // tiles' bytes, and their products are never read.
            const uint32_t id = tc::instr_desc(0, 128, 0) | static_cast<uint32_t>(q.bn >> 3) << 17;
            int s = 0, b = 0, r = 0;
            uint32_t phase = 0, tphase = 1, sphase = 0;
            bool ok = true;
            for (int g = g0; g < g1; g++) {
                // the scales too, for the epilogue, which then waits for the products alone
                if (!wait_phase(full(s), phase) || !wait_phase(sfull(r), sphase) || !wait_phase(tempty(b), tphase)) ok = false;
                if (!__all_sync(0xffffffffu, ok)) { report(p); break; }
                tc::fence_after_sync();
                if (elect_one()) {
                    mma_group<1>(tmem + b * q.bn, ring + s * q.rows * BK, wring + s * q.bn * BK, id);
                    tc::commit(empty(s));
                    tc::commit(tfull(b));
                }
                __syncwarp();
                if (++s == q.stages) { s = 0; phase ^= 1; }
                if (++b == q.nbuf) { b = 0; tphase ^= 1; }
                if (++r == C::SR) { r = 0; sphase ^= 1; }
            }
            finished(empty(0), q.stages, s, phase, tfull(0), q.nbuf, b, tphase, p);
        } else if (warp == 2 && rank != p.stalled) {
            int r = 0;
            uint32_t phase = 1;
            const float *sa = p.sa + (m0 + lane) * p.sa_row + g0 * p.sa_group;
            const float *sw = p.sw + (n0 / 128 + (lane < 3 ? lane : 0)) * p.sw_row + g0 * p.sw_group;
            const bool w_in = lane < 3 && (n0 / 128 + lane) * 128 < min(p.N, n0 + q.bn);
            for (int g = g0; g < g1; g++) {
                if (!wait_phase(sempty(r), phase)) { report(p); break; }
                const uint32_t at = tc::smem_addr(scales + r * C::SLOT);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (lane + 32 * j < rows) cp_async4(at + (lane + 32 * j) * 4, sa + 32 * j * p.sa_row);
                if (w_in) cp_async4(at + (128 + lane) * 4, sw);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(sfull(r)) : "memory");
                sa += p.sa_group;
                sw += p.sw_group;
                if (++r == C::SR) { r = 0; phase ^= 1; }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::REGS_EPILOGUE));
        const int quarter = warp % 4, first = (warp - 4) / 4 * per;
        const int mine = max(0, min(per, chunks - first));
        const int row = quarter * 32 + lane;
        float acc[MAXC][16];
#pragma unroll
        for (int c = 0; c < MAXC; c++)
#pragma unroll
            for (int j = 0; j < 16; j++) acc[c][j] = 0.f;
        bool ok = true;
        if (mine > 0 && quarter * 32 < rows) {
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + first * 16;
            int b = 0, r = 0;
            uint32_t tphase = 0;
            // which block of W's scales a chunk has
            int block[MAXC];
#pragma unroll
            for (int c = 0; c < MAXC; c++) block[c] = (n0 + (first + c) * 16) / 128 - n0 / 128;
            for (int g = g0; g < g1; g++) {
                if (!wait_warp(tfull(b), tphase)) { ok = false; break; }
                tc::fence_after_sync();
                const float *slot = scales + r * C::SLOT;
                const float s = slot[row];
                constexpr int AT_ONCE = MAXC < 2 ? MAXC : 2;   // chunks in flight: registers
#pragma unroll
                for (int c = 0; c < MAXC; c += AT_ONCE) {
                    float v[AT_ONCE][16], f[AT_ONCE];
#pragma unroll
                    for (int k = 0; k < AT_ONCE; k++)
                        if (c + k < mine) {
                            tc::tmem_ld16(lanes + b * q.bn + (c + k) * 16, v[k]);
                            f[k] = s * slot[128 + block[c + k]];
                        }
                    tc::tmem_ld_wait();
                    if (c + AT_ONCE >= MAXC) {
                        tc::fence_before_sync();
                        __syncwarp();   // every lane has read the slot
                        if (lane == 0) {
                            arrive_local(tempty(b));
                            arrive_local(sempty(r));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < AT_ONCE; k++)
                        if (c + k < mine)
#pragma unroll
                            for (int j = 0; j < 16; j++) acc[c + k][j] = fmaf(v[k][j], f[k], acc[c + k][j]);
                }
                if (++b == q.nbuf) { b = 0; tphase ^= 1; }
                if (++r == C::SR) r = 0;
            }
            if (!ok) {
                report(p);
                *reinterpret_cast<volatile uint32_t *>(dyn + C::FAILED) = 1;
            }
            if (ok && row < rows)
#pragma unroll
                for (int c = 0; c < MAXC; c++)
                    if (c < mine) {
                        if (q.split == 1) {
                            store16(p, m0 + row, n0 + (first + c) * 16, acc[c]);
                        } else {
                            // the ring again, now that this CTA's last MMA is done; an odd pitch spreads the banks
                            float *red = reinterpret_cast<float *>(dyn) + row * (q.bn + 1) + (first + c) * 16;
#pragma unroll
                            for (int j = 0; j < 16; j++) red[j] = acc[c][j];
                        }
                    }
        }
    }
    if (q.split > 1) {
        cluster_sync();
        if (warp >= 4) slim_join(p.out, p.ld_out, p.out_dtype, min(q.bn, p.N - n0), q.bn, q.split, ring, m0, n0, rows, rank);
        cluster_sync();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc<512>(tmem);
}

// ---- many rows of A -----------------------------------------------------------------------

struct Wide {
    static constexpr int EW = 16;                    // epilogue warps: four for each quarter of the TMEM lanes
    static constexpr int COLS = 256 * 4 / EW;        // columns of the tile per epilogue thread
    static constexpr int THREADS = 128 + EW * 32;    // copies, MMAs, scales, one idle warp, then the epilogue's
    // registers per thread: 640 * 96 at launch = 128 * 32 + 512 * 112
    static constexpr int REGS_CONTROL = 32, REGS_EPILOGUE = 112;
    static constexpr int STAGE = 2 * 128 * BK;       // per CTA: its 128 rows of A and its 128 rows of W
    static constexpr int STAGES = 5;
    static constexpr int BOX = 32 * 128;             // an epilogue warp's outputs on their way to memory: 32 rows of 128 bytes
    static constexpr int SR = 2;                     // slots of scales, two groups each: 128 rows' and the tile's two of W
    static constexpr int SLOT = 132 * 2;             // floats: [128 rows, 2 blocks of W][2 groups]
    static constexpr int SCALES = SR * SLOT * 4;
    static constexpr int BARS = (2 * STAGES + 4 + 2 * SR) * 8;
    static constexpr int SMEM = STAGES * STAGE + EW * BOX + SCALES + BARS + 16;
};
static_assert(Wide::SMEM <= 227 * 1024, "shared memory of one CTA");

struct Tiles {
    int m, n;          // tiles of 256
    int band;          // tiles of A that are walked together over all of W, so that W stays in L2
};

__device__ __forceinline__ void tile_at(const Tiles &t, int i, int *tm, int *tn)
{
    const int per = t.band * t.n, b = i / per, r = i % per;
    const int h = min(t.band, t.m - b * t.band);
    *tm = b * t.band + r % h;
    *tn = r / h;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide::THREADS, 1)
wide_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
            const __grid_constant__ CUtensorMap tm_out, const int tma_n, const Fp8Params p, const Tiles tiles)
{
    using C = Wide;
    extern __shared__ __align__(1024) unsigned char dyn[];
    const uint32_t ring = tc::smem_addr(dyn);
    float *scales = reinterpret_cast<float *>(dyn + C::STAGES * C::STAGE + C::EW * C::BOX);   // [SR][128 | 2]
    const uint32_t b0 = tc::smem_addr(scales) + C::SCALES;
    volatile uint32_t *tmem_base = reinterpret_cast<uint32_t *>(dyn + C::SMEM - 16);
    auto full = [&](int s) { return b0 + s * 8; };
    auto empty = [&](int s) { return b0 + (C::STAGES + s) * 8; };
    auto tfull = [&](int b) { return b0 + (2 * C::STAGES + b) * 8; };
    auto tempty = [&](int b) { return b0 + (2 * C::STAGES + 2 + b) * 8; };
    auto sfull = [&](int r) { return b0 + (2 * C::STAGES + 4 + r) * 8; };
    auto sempty = [&](int r) { return b0 + (2 * C::STAGES + 4 + C::SR + r) * 8; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; s++) { tc::mbar_init(full(s), 1); tc::mbar_init(empty(s), 1); }
        for (int b = 0; b < 2; b++) { tc::mbar_init(tfull(b), 1); tc::mbar_init(tempty(b), 2 * C::EW); }
        for (int r = 0; r < C::SR; r++) { tc::mbar_init(sfull(r), 32); tc::mbar_init(sempty(r), C::EW); }
        tc::prefetch_tensormap(&tm_w);
        tc::prefetch_tensormap(&tm_a);
        if (tma_n > 0) tc::prefetch_tensormap(&tm_out);
    }
    pdl_wait();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(b0 + C::BARS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    pdl_release();

    const uint32_t tmem = *tmem_base;
    const int groups = (p.K + BK - 1) / BK;
    const int total = tiles.m * tiles.n, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::REGS_CONTROL));
        if (warp == 0) {
            if (lane == 0) {
                int s = 0;
                uint32_t phase = 1;
                bool ok = true;
                for (int i = pair; i < total && ok; i += pairs) {
                    int tm, tn;
                    tile_at(tiles, i, &tm, &tn);
                    const int m0 = tm * 256 + rank * 128, n0 = tn * 256 + rank * 128;
                    for (int g = 0; g < groups; g++) {
                        if (!wait_phase(empty(s), phase)) { report(p); ok = false; break; }
                        // both CTAs' copies are counted on the barrier of the one that issues the MMAs
                        if (rank == 0) tc::mbar_expect_tx(full(s), 2 * C::STAGE);
                        const uint32_t at = ring + s * C::STAGE, bar = in_cta(full(s), 0);
                        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                                     " [%0], [%1, {%2, %3}], [%4];" :: "r"(at), "l"(&tm_a), "r"(g * BK), "r"(m0), "r"(bar) : "memory");
                        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                                     " [%0], [%1, {%2, %3}], [%4];" :: "r"(at + 128 * BK), "l"(&tm_w), "r"(g * BK), "r"(n0), "r"(bar) : "memory");
                        if (++s == C::STAGES) { s = 0; phase ^= 1; }
                    }
                }
                // the last arrivals on this CTA's barriers come from the pair's other CTA: not before them does it end
                int k = s;
                uint32_t parity = phase;
                for (int i = 0; i < C::STAGES && ok; i++) {
                    if (!wait_phase(empty(k), parity)) { report(p); ok = false; }
                    if (++k == C::STAGES) { k = 0; parity ^= 1; }
                }
                // Where something gave up, both CTAs' copies: a stage of which only one CTA has issued its half lets this
                // wait run out too, long after what was issued has landed.
                if (!ok && rank == 0) landed(full(0), C::STAGES, s, phase, p);
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0) {
                constexpr uint32_t ID = tc::instr_desc(0, 256, 256);
                int s = 0, b = 0;
                uint32_t phase = 0, tphase = 1;
                bool ok = true;
                for (int i = pair; i < total && ok; i += pairs)
                    for (int g = 0; g < groups; g++) {
                        // the accumulator last: what follows it is on the way from one group to the next
                        if (!wait_phase(full(s), phase) || !wait_phase(tempty(b), tphase)) ok = false;
                        if (!__all_sync(0xffffffffu, ok)) { report(p); ok = false; break; }
                        tc::fence_after_sync();
                        const uint32_t at = ring + s * C::STAGE;
                        if (elect_one()) {
                            mma_group<2>(tmem + b * 256, at, at + 128 * BK, ID);
                            commit_pair(empty(s));
                            commit_pair(tfull(b));
                        }
                        __syncwarp();
                        if (++s == C::STAGES) { s = 0; phase ^= 1; }
                        if (++b == 2) { b = 0; tphase ^= 1; }
                    }
                finished(empty(0), C::STAGES, s, phase, tfull(0), 2, b, tphase, p);
            }
            __syncwarp();
        } else if (warp == 2 && static_cast<int>(rank) != p.stalled) {
            // the groups' scales, copied while the tensor core is groups behind
            int r = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int i = pair; i < total && ok; i += pairs) {
                int tm, tn;
                tile_at(tiles, i, &tm, &tn);
                const int m0 = tm * 256 + rank * 128 + lane, nb = tn * 2;
                const float *sa = p.sa + m0 * p.sa_row, *sw = p.sw + (nb + (lane & 1)) * p.sw_row;
                const bool w_in = lane < 2 && (nb + lane) * 128 < p.N;
                for (int g = 0; g < groups; g += 2) {
                    if (!wait_phase(sempty(r), phase)) { report(p); ok = false; break; }
                    const uint32_t at = tc::smem_addr(scales + r * C::SLOT);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (g + h < groups) {
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                if (m0 + 32 * j < p.M) cp_async4(at + ((lane + 32 * j) * 2 + h) * 4, sa + 32 * j * p.sa_row);
                            if (w_in) cp_async4(at + ((128 + lane) * 2 + h) * 4, sw);
                        }
                        sa += p.sa_group;
                        sw += p.sw_group;
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(sfull(r)) : "memory");
                    if (++r == C::SR) { r = 0; phase ^= 1; }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::REGS_EPILOGUE));
        const int quarter = warp % 4, c0 = (warp - 4) / 4 * C::COLS;      // TMEM lanes, columns of the tile
        const int row = quarter * 32 + lane;
        unsigned char *box = dyn + C::STAGES * C::STAGE + (warp - 4) * C::BOX;
        int b = 0, r = 0;
        uint32_t tphase = 0, sphase = 0;
        bool ready = false;
        for (int i = pair; i < total; i += pairs) {
            float2 acc[C::COLS / 2];
#pragma unroll
            for (int c = 0; c < C::COLS / 2; c++) acc[c] = make_float2(0.f, 0.f);
            bool ok = true;
            float2 s2;
            for (int g = 0; g < groups; g++) {
                if (g % 2 == 0) {
                    // two groups' scales at a time
                    if (!wait_warp(sfull(r), sphase)) { ok = false; break; }
                    const float2 *slot = reinterpret_cast<const float2 *>(scales + r * C::SLOT);
                    const float2 x = slot[row], y = slot[128 + c0 / 128];
                    s2 = make_float2(x.x * y.x, x.y * y.y);
                    __syncwarp();
                    if (lane == 0) arrive_local(sempty(r));
                    if (++r == C::SR) { r = 0; sphase ^= 1; }
                }
                const float2 f = g % 2 == 0 ? make_float2(s2.x, s2.x) : make_float2(s2.y, s2.y);
                if (!ready && !wait_warp(tfull(b), tphase)) { ok = false; break; }
                tc::fence_after_sync();
                const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * 256 + c0;
                uint32_t v[32];
                tmem_ld32(at, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; j++)
                    acc[j] = ffma2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), f, acc[j]);
                tmem_ld32(at + 32, v);
                tc::tmem_ld_wait();
                tc::fence_before_sync();
                if (lane == 0) arrive_cluster(in_cta(tempty(b), 0));
                if (++b == 2) { b = 0; tphase ^= 1; }
                // asked here, answered by the time the sums below are done
                ready = __all_sync(0xffffffffu, test_phase(tfull(b), tphase));
#pragma unroll
                for (int j = 0; j < 16; j++)
                    acc[16 + j] = ffma2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), f, acc[16 + j]);
            }
            if (!ok) { report(p); break; }
            int tm, tn;
            tile_at(tiles, i, &tm, &tn);
            const int m0 = tm * 256 + rank * 128 + quarter * 32, n0 = tn * 256 + c0;   // of this warp's box
            if (m0 >= p.M || n0 >= p.N) continue;
            if (n0 < tma_n) {
                // 32 rows of 128 bytes with the map's swizzle (16-byte piece j of row l at j ^ (l % 8)),
                // written by TMA, which leaves out what lies past the matrix
                auto put = [&](const uint32_t (&w)[32], int x) {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        *reinterpret_cast<uint4 *>(box + lane * 128 + ((j ^ (lane % 8)) * 16)) =
                            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                                     :: "l"(&tm_out), "r"(x), "r"(m0), "r"(tc::smem_addr(box)) : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                };
                if (p.out_dtype == 2) {
#pragma unroll
                    for (int h = 0; h < C::COLS / 32; h++) {
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            w[2 * j] = __float_as_uint(acc[16 * h + j].x);
                            w[2 * j + 1] = __float_as_uint(acc[16 * h + j].y);
                        }
                        if (n0 + 32 * h < p.N) put(w, n0 + 32 * h);
                    }
                } else {
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        w[j] = p.out_dtype == 0 ? pack_bf16x2(acc[j].x, acc[j].y) : tc::pack_f16x2(acc[j].x, acc[j].y);
                    put(w, n0);
                }
            } else if (m0 + lane < p.M) {
#pragma unroll
                for (int c = 0; c < C::COLS; c++)
                    if (n0 + c < p.N)
                        store_out(p.out, static_cast<int64_t>(m0 + lane) * p.ld_out + n0 + c, p.out_dtype, c % 2 ? acc[c / 2].y : acc[c / 2].x);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc::fence_before_sync();
    cluster_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

// ---- any strides and alignments -----------------------------------------------------------

// e4m3 -> fp32 (exact)
__device__ __forceinline__ float e4m3_to_f32(uint8_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

constexpr int GT = 64, GK = 32;
__global__ void __launch_bounds__(256, 3) general_kernel(const Fp8Params p, int tiles_n)
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

// ---- host ---------------------------------------------------------------------------------

// cuTensorMapEncodeTiled, fetched once through the runtime
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// A map over `rows` rows of `cols` elements of `es` bytes at a pitch of `ld` elements, moved in
// boxes of `box` rows x 128 bytes with the 128-byte swizzle.
cudaError_t encode(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t ld, int box,
                   CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8, int es = 1)
{
    const auto enc = encoder();
    if (!enc) return cudaErrorSymbolNotFound;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box)};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = enc(m, type, 2, const_cast<void *>(base), dims, strides, boxes, steps,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// TMA's conditions; a single row has no pitch of its own.
bool tma_rows(const void *base, int64_t *ld, int64_t rows, int64_t cols)
{
    if (rows == 1) *ld = (cols + 15) / 16 * 16;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && *ld % 16 == 0 && *ld < (int64_t(1) << 39);
}

// A launch with programmatic stream serialization over clusters of `split` CTAs.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    Launch(dim3 grid, int threads, int smem, int split, cudaStream_t stream)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = split > 1 ? 2 : 1;
    }
};

// How many CTAs of a kernel run at once in clusters of 1 .. 8 (clusters leave SMs unused that do not
// fit their GPC), asked once.
struct Fit {
    int ctas[9] = {};
    template <typename K>
    cudaError_t ask(K kernel, int threads, int smem, int sms, int per_sm)
    {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        ctas[1] = sms * per_sm;
        for (int split = 2; split <= 8 && e == cudaSuccess; split++) {
            Launch l(dim3(split), threads, smem, split, nullptr);
            l.at[0] = l.at[1];   // the cluster alone
            l.cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg);
            ctas[split] = n * split;
        }
        return e;
    }
};

// The plans are compared by their time in nanoseconds, from what was measured for N of 1024 to 20512,
// K of 1024 to 8192 and M of 16 to 512 with every split (the choice is within 10% of the best of
// them): start and end of a wave of CTAs, then its groups of 128 k, each by the slower of the epilogue and the
// streams (5.7 kB/ns from HBM over all SMs), then the join of a split.
double plan_time(int64_t ctas, int fit, int groups, int split, double start, double step, double join)
{
    const double waves = static_cast<double>((ctas + fit - 1) / fit);
    return waves * (start + step * ((groups + split - 1) / split)) + (split > 1 ? join : 0.);
}

// The split of least time.
template <int NT>
double plan_thin(const Fp8Params &p, const Fit &fit, int *split)
{
    using C = Thin<NT>;
    const int groups = (p.K + BK - 1) / BK, tiles_n = (p.N - 1) / 128 + 1, tiles_t = (p.M + NT - 1) / NT;
    double least = 1e30;
    for (int k = 1; k <= 8 && k <= groups; k++) {
        if (fit.ctas[k] == 0) continue;
        const int64_t ctas = static_cast<int64_t>(tiles_n) * tiles_t * k;
        const double at_once = ctas < fit.ctas[k] ? ctas : fit.ctas[k], hbm = at_once * 128 * BK / tiles_t / 5700.;
        const double l2 = (at_once > fit.ctas[1] / 2 ? 2 : 1) * C::STAGE / 85.;      // a group's copies of one SM's CTAs, fitted
        double step = NT > 32 ? 322. : NT > 16 ? 288. : 281.;
        if (step < hbm) step = hbm;
        if (step < l2) step = l2;
        const double t = plan_time(ctas, fit.ctas[k], groups, k, NT > 32 ? 4000. : NT > 16 ? 3200. : 2700., step, 1100.);
        if (t < least) { least = t; *split = k; }
    }
    return least;
}

template <int NT>
cudaError_t run_thin(const Fp8Params &p, int split, int64_t ld_a, int64_t ld_w, cudaStream_t stream)
{
    using C = Thin<NT>;
    CUtensorMap tw, ta;
    cudaError_t e;
    if ((e = encode(&tw, p.w, p.K, p.N, ld_w, 128)) != cudaSuccess) return e;
    if ((e = encode(&ta, p.a, p.K, p.M, ld_a, NT)) != cudaSuccess) return e;
    Launch l(dim3(static_cast<unsigned>((p.N - 1) / 128 + 1) * split, static_cast<unsigned>((p.M + NT - 1) / NT)), C::THREADS, C::SMEM, split,
             stream);
    return cudaLaunchKernelEx(&l.cfg, thin_kernel<NT>, ta, tw, p, split);
}

constexpr int SLIM_SMEM = Slim::RING + Slim::TAIL;

// The plan of least time among the splits, each with the tile of W that fills the GPU once.
double plan_slim(const Fp8Params &p, const Fit &fit, SlimPlan *best)
{
    const int groups = (p.K + BK - 1) / BK, mt = (p.M + 127) / 128;
    const int rows = p.M >= 128 ? 128 : (p.M + 7) / 8 * 8;
    double least = 1e30;
    if (mt > 65535) return least;                   // the grid's y axis ends there
    for (int split = 1; split <= 8 && split <= groups; split++) {
        if (fit.ctas[split] == 0) continue;
        const int tiles = fit.ctas[split] / (split * mt);           // of W in one wave
        int bn = tiles < 1 ? p.N : (p.N - 1) / tiles + 1;
        bn = bn > 256 ? 256 : (bn + 15) / 16 * 16;
        if (split > 1 && (bn + 1) * rows * 4 > Slim::RING) continue;
        const int64_t ctas = static_cast<int64_t>((p.N - 1) / bn + 1) * split * mt;
        const double t = plan_time(ctas, fit.ctas[split], groups, split, 3400., 250. + 2.05 * bn, 1300. + 0.125 * rows * bn);
        if (t < least) {
            least = t;
            best->bn = bn;
            best->split = split;
        }
    }
    best->rows = rows;
    const int s = Slim::RING / ((rows + best->bn) * BK), n = 512 / best->bn;
    best->stages = s < Slim::MAX_STAGES ? s : Slim::MAX_STAGES;
    best->nbuf = n < Slim::MAX_BUF ? n : Slim::MAX_BUF;
    return least;
}

template <int MAXC>
cudaError_t run_slim(const Fp8Params &p, const SlimPlan &q, int64_t ld_a, int64_t ld_w, cudaStream_t stream)
{
    CUtensorMap tw, ta;
    cudaError_t e;
    if ((e = encode(&tw, p.w, p.K, p.N, ld_w, q.bn)) != cudaSuccess) return e;
    if ((e = encode(&ta, p.a, p.K, p.M, ld_a, q.rows)) != cudaSuccess) return e;
    Launch l(dim3(static_cast<unsigned>((p.N - 1) / q.bn + 1) * q.split, static_cast<unsigned>((p.M + 127) / 128)), Slim::THREADS,
             SLIM_SMEM, q.split, stream);
    return cudaLaunchKernelEx(&l.cfg, slim_kernel<MAXC>, ta, tw, p, q);
}

cudaError_t run_wide(const Fp8Params &p, int64_t ld_a, int64_t ld_w, int sms, cudaStream_t stream)
{
    CUtensorMap tw, ta, to = {};
    cudaError_t e;
    if ((e = encode(&tw, p.w, p.K, p.N, ld_w, 128)) != cudaSuccess) return e;
    if ((e = encode(&ta, p.a, p.K, p.M, ld_a, 128)) != cudaSuccess) return e;
    const int es = p.out_dtype == 2 ? 4 : 2;
    const bool tma_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ld_out * es % 16 == 0 && p.ld_out < (int64_t(1) << 38);
    const CUtensorMapDataType type = p.out_dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : p.out_dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    // TMA writes whole 16-byte pieces, also where the map ends inside one: then a warp's last columns are stored without
    // it (both ways for every warp are 2.37 ms against 2.19 at the widest product: registers)
    const int tma_n = !tma_out ? 0 : static_cast<int64_t>(p.N) * es % 16 == 0 ? p.N : p.N / Wide::COLS * Wide::COLS;
    if (tma_n > 0 && (e = encode(&to, p.out, p.N, p.M, p.ld_out, 32, type, es)) != cudaSuccess) return e;
    // the pairs at work share two tiles of W: 2.15 ms at the widest product, 2.25 in bands of 8, 2.31 in bands of 64
    const Tiles t{(p.M - 1) / 256 + 1, (p.N - 1) / 256 + 1, sms / 4};
    const int64_t total = static_cast<int64_t>(t.m) * t.n;
    if (total > INT32_MAX - 4096) return cudaErrorInvalidConfiguration;
    const int pairs = static_cast<int>(total < sms / 2 ? total : sms / 2);
    return launch_pdl(wide_kernel, dim3(2 * pairs), dim3(Wide::THREADS), Wide::SMEM, stream, ta, tw, to, tma_n, p, t);
}

// What the launches need to know of a device, and the kernels' shared-memory limits set there, once.
struct Device {
    int sms = 0;
    Fit thin16, thin32, thin64, slim;
    cudaError_t ask(int dev)
    {
        cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        const auto limit = [](auto kernel, int smem) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        };
        if (e == cudaSuccess) e = thin16.ask(thin_kernel<16>, Thin<16>::THREADS, Thin<16>::SMEM, sms, 2);
        if (e == cudaSuccess) e = thin32.ask(thin_kernel<32>, Thin<32>::THREADS, Thin<32>::SMEM, sms, 2);
        if (e == cudaSuccess) e = thin64.ask(thin_kernel<64>, Thin<64>::THREADS, Thin<64>::SMEM, sms, 2);
        if (e == cudaSuccess) e = slim.ask(slim_kernel<4>, Slim::THREADS, SLIM_SMEM, sms, 1);
        if (e == cudaSuccess) e = limit(slim_kernel<1>, SLIM_SMEM);
        if (e == cudaSuccess) e = limit(slim_kernel<2>, SLIM_SMEM);
        if (e == cudaSuccess) e = limit(wide_kernel, Wide::SMEM);
        return e;
    }
};

// Kept once it has been asked with success: a failure is the call's, not the process's.
cudaError_t this_device(const Device **out)
{
    constexpr int MOST = 64;
    static Device devices[MOST];
    static std::atomic<bool> known[MOST];
    static std::mutex asking;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= MOST) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        const std::lock_guard<std::mutex> one(asking);
        if (!known[dev].load(std::memory_order_relaxed)) {
            const cudaError_t asked = devices[dev].ask(dev);
            if (asked != cudaSuccess) return asked;
            known[dev].store(true, std::memory_order_release);
        }
    }
    *out = &devices[dev];
    return cudaSuccess;
}

// Which kernel a call takes, in what tiles.
struct Choice {
    int rows = 0;              // of A per tile: 0 (general_kernel), 16, 32, 64 (thin_kernel), 128 (slim_kernel), 256 (wide_kernel)
    int split = 1;
    SlimPlan slim;
    int64_t ld_a, ld_w;
    const Device *device = nullptr;
};

cudaError_t choose(const Fp8Params &p, Choice *c)
{
    c->ld_a = p.ld_a;
    c->ld_w = p.ld_w;
    if (p.K == 0 || !tma_rows(p.a, &c->ld_a, p.M, p.K) || !tma_rows(p.w, &c->ld_w, p.N, p.K)) return cudaSuccess;
    const cudaError_t e = this_device(&c->device);
    if (e != cudaSuccess) return e;
    const Device *d = c->device;
    if (p.M <= 32) {
        c->rows = p.M <= 16 ? 16 : 32;
        p.M <= 16 ? plan_thin<16>(p, d->thin16, &c->split) : plan_thin<32>(p, d->thin32, &c->split);
        return cudaSuccess;
    }
    // More rows: the arrangement of least time. Beyond a thousand rows that is slim_kernel where few columns
    // or a short inner axis leave the pairs of wide_kernel idle or starting: 1311 x 167 x 365 4.0 us against 6.7,
    // 1968 x 600 x 684 7.0 against 9.1, 1500 x 4096 x 4096 33.4 against 35.4.
    const double slim = plan_slim(p, d->slim, &c->slim);
    if (p.M <= 64 && plan_thin<64>(p, d->thin64, &c->split) <= slim) {
        c->rows = 64;
        return cudaSuccess;
    }
    const int groups = (p.K + BK - 1) / BK;
    const int64_t tiles = (static_cast<int64_t>(p.M) + 255) / 256 * ((static_cast<int64_t>(p.N) + 255) / 256);
    const int pairs = d->sms / 2;
    const double busy = tiles < pairs ? static_cast<double>(tiles) / pairs : 1.;
    const bool wide = 6000. + (340. + 100. * busy) * groups * static_cast<double>((tiles + pairs - 1) / pairs) < slim;
    c->rows = wide ? 256 : 128;
    c->split = wide ? 1 : c->slim.split;
    return cudaSuccess;
}

}  // namespace

cudaError_t plan_fp8_matmul(const Fp8Params &p, int32_t (&plan)[3])
{
    Choice c;
    const cudaError_t e = choose(p, &c);
    if (e != cudaSuccess) return e;
    plan[0] = c.rows;
    plan[1] = c.split;
    plan[2] = c.rows == 0 ? GT : c.rows <= 64 ? 128 : c.rows == 128 ? c.slim.bn : 256;
    return cudaSuccess;
}

cudaError_t launch_fp8_matmul(const Fp8Params &p, cudaStream_t stream)
{
    Choice c;
    const cudaError_t e = choose(p, &c);
    if (e != cudaSuccess) return e;
    switch (c.rows) {
    case 16: return run_thin<16>(p, c.split, c.ld_a, c.ld_w, stream);
    case 32: return run_thin<32>(p, c.split, c.ld_a, c.ld_w, stream);
    case 64: return run_thin<64>(p, c.split, c.ld_a, c.ld_w, stream);
    case 128: {
        const int per = (c.slim.bn / 16 + 3) / 4;
        if (per <= 1) return run_slim<1>(p, c.slim, c.ld_a, c.ld_w, stream);
        if (per <= 2) return run_slim<2>(p, c.slim, c.ld_a, c.ld_w, stream);
        return run_slim<4>(p, c.slim, c.ld_a, c.ld_w, stream);
    }
    case 256: return run_wide(p, c.ld_a, c.ld_w, c.device->sms, stream);
    }
    const int64_t tm = (static_cast<int64_t>(p.M) + GT - 1) / GT, tn = (static_cast<int64_t>(p.N) + GT - 1) / GT;
    if (tm * tn > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(general_kernel, dim3(static_cast<unsigned>(tm * tn)), dim3(256), 0, stream, p, static_cast<int>(tn));
}

}  // namespace kda
