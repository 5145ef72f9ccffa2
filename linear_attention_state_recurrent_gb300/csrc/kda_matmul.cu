// kda_matmul: out = act(A W^T + bias) + residual, bf16 or fp16 operands, fp32 sums.
//
// The sums of a tile stay in tensor memory over the whole inner axis; the epilogue reads them once, adds the bias, applies
// the activation, adds the residual and rounds once. TMA brings 128-byte-wide tiles (64 of the inner axis) with the 128-byte
// swizzle that the matrix descriptors name; what lies past the matrices reads as zeros. Two arrangements:
//  - tile_kernel: 128 rows of W are the MMA's M side, 16 to 128 rows of A its N side, two CTAs an SM. The inner axis may be
//    split over a cluster whose CTAs join their sums through distributed shared memory in a fixed order. For few rows of A, bound
//    by the stream of weights, and for products that do not fill the GPU with the tiles of
//  - pair_kernel: 256 x 256 by a pair of CTAs (cta_group::2), persistent, two accumulators, so that a tile's epilogue is beside the
//    next one's MMAs; outputs and residuals move by TMA.
// Operands that TMA cannot address (rows off 16-byte boundaries) go through tile_kernel with warps that load them element by element
// into the same layout.
#include <atomic>
#include <climits>
#include <mutex>
#include <type_traits>
#include <cuda_fp16.h>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_matmul.h"
#include "kda_mma.cuh"
#include "kda_pdl.cuh"

namespace kda {
namespace {

using namespace mma;

constexpr int BK = 64;                         // of the inner axis per stage: 128 bytes a row

// Matrix descriptor of a K-major tile of 128-byte rows with the 128-byte swizzle; the next 16 of the inner axis are 32 bytes on.
__device__ __forceinline__ uint64_t desc(uint32_t at)
{
    constexpr uint32_t HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
    return static_cast<uint64_t>(HIGH) << 32 | (1u << 16) | (at >> 4);
}
// d (+)= a b^T over one stage
template <int CG>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
#pragma unroll
    for (int k = 0; k < BK / 16; k++) {
        const uint32_t acc = add || k > 0;
        if (CG == 1)
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                         :: "r"(d), "l"(desc(a + k * 32)), "l"(desc(b + k * 32)), "r"(idesc), "r"(acc));
        else
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                         :: "r"(d), "l"(desc(a + k * 32)), "l"(desc(b + k * 32)), "r"(idesc), "r"(acc));
    }
}
__device__ __forceinline__ void commit_pair(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(mbar), "h"(static_cast<uint16_t>(3)) : "memory");
}

// Waits for a barrier's phase; gives up after 4e9 clocks (~2 s).
__device__ __noinline__ bool wait_on(uint32_t mbar, uint32_t parity)
{
    const long long start = clock64();
    while (!phase_over(mbar, parity))
        if (clock64() - start > 4000000000ll) return false;
    return true;
}
__device__ __forceinline__ bool wait(uint32_t mbar, uint32_t parity) { return phase_over(mbar, parity) || wait_on(mbar, parity); }
__device__ __forceinline__ bool wait_warp(uint32_t mbar, uint32_t parity) { return __all_sync(0xffffffffu, wait(mbar, parity)); }
__device__ __forceinline__ void report(const MatmulParams &p)
{
    if (p.err) atomicOr(p.err, kErrTimeout);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}

// ---- elements -----------------------------------------------------------------------------

__device__ __forceinline__ float load_as(const void *p, int64_t i, int dtype)
{
    if (dtype == KDA_BF16) return bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
    if (dtype == KDA_FP16) return __half2float(static_cast<const __half *>(p)[i]);
    return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_as(void *p, int64_t i, int dtype, float v)
{
    if (dtype == KDA_BF16) static_cast<uint16_t *>(p)[i] = f32_to_bf16(v);
    else if (dtype == KDA_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// y / (1 + e^-x), by e^-|x|: the divisor is at most 2 (from 2^126 on, x below -87, the quotient to two steps would be 0).
__device__ __forceinline__ float gated(float y, float x)
{
    const float e = expf(-fabsf(x));
    return __fdividef(x < 0.f ? y * e : y, 1.f + e);
}

// The activation over values held in registers. The one branch is around all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act)
{
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = f(v[i]);
    };
    switch (act) {
    case KDA_ACT_RELU: each([](float x) { return x < 0.f ? 0.f : x; }); break;   // a NaN stays one
    // (a quotient to two steps: the exact one takes a slow path where e^-x is large, 36 us for 24 at 128 x 12,288 x 4096)
    case KDA_ACT_SILU: each([](float x) { return gated(x, x); }); break;
    case KDA_ACT_SIGMOID: each([](float x) { return gated(1.f, x); }); break;
    case KDA_ACT_GELU: each([](float x) { return 0.5f * x * erfcf(-0.70710678118654752f * x); }); break;
    // x (1 + tanh u) / 2 = x / (1 + e^{-2u}), u = (2 / pi)^(1/2) (x + 0.044715 x^3)
    case KDA_ACT_GELU_TANH: each([](float x) { return gated(x, 1.5957691216057308f * (x + 0.044715f * x * x * x)); }); break;
    }
}

// The residuals of outputs m .. m + 15 of column n.
__device__ __forceinline__ void fetch(const MatmulParams &p, float (&r)[16], int m, int n)
{
#pragma unroll
    for (int i = 0; i < 16; i++) r[i] = p.res && n < p.N && m + i < p.M ? load_as(p.res, static_cast<int64_t>(m + i) * p.ld_res + n, p.out_dtype) : 0.f;
}
// Outputs m .. m + 15 of column n, from their sums.
__device__ __forceinline__ void finish(const MatmulParams &p, float (&v)[16], const float (&r)[16], int m, int n)
{
    if (n >= p.N) return;
    if (p.bias) {
        const float b = load_as(p.bias, n, p.bias_dtype);
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] += b;
    }
    activate(v, p.act);
    if (p.res) {
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] += r[i];
    }
#pragma unroll
    for (int i = 0; i < 16; i++)
        if (m + i < p.M) store_as(p.out, static_cast<int64_t>(m + i) * p.ld_out + n, p.out_dtype, v[i]);
}

// ---- tiles of 128 rows of W by NT rows of A -------------------------------------------------

// LOOSE: operands on any boundaries, loaded by eight warps more.
template <int NT, bool LOOSE>
struct Tile {
    static constexpr int EW = 8;                                    // epilogue warps: two for each quarter of the TMEM lanes
    static constexpr int THREADS = (2 + EW + (LOOSE ? 8 : 0)) * 32; // copies, MMAs, the epilogue's, and the loose operands' copies
    static constexpr int STAGE = 128 * 128 + NT * 128;
    static constexpr int TWO = 113 * 1024 / STAGE, ONE = 226 * 1024 / STAGE < 10 ? 226 * 1024 / STAGE : 10;   // stages with two CTAs per SM, with one
    static constexpr int COLS = NT < 32 ? 32 : NT;                  // of tensor memory
};

template <int NT, bool LOOSE>
__global__ void __launch_bounds__(Tile<NT, LOOSE>::THREADS, LOOSE ? 1 : 2)
tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ MatmulParams p, const int split, const int stages)
{
    using T = Tile<NT, LOOSE>;
    static_assert(NT * 132 * 4 <= T::TWO * T::STAGE, "a split's sums, in the ring once it is drained");
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ uint64_t bars[2 * T::ONE + 1];
    __shared__ uint32_t tmem_at, failed;
    const uint32_t s0 = tc::smem_addr(sm), b0 = tc::smem_addr(bars);
    auto full = [&](int s) { return b0 + s * 8; };
    auto empty = [&](int s) { return b0 + (T::ONE + s) * 8; };
    const uint32_t done = b0 + 2 * T::ONE * 8;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % split, n0 = blockIdx.x / split * 128, m0 = blockIdx.y * NT;
    const int steps = (p.K + BK - 1) / BK;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * rank / split), k1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / split);
    auto load = [&](int k, int s) {
        const uint32_t at = s0 + s * T::STAGE;
        tc::mbar_expect_tx(full(s), T::STAGE);
        tc::tma_load_2d(at, &tm_w, k * BK, n0, full(s));
        tc::tma_load_2d(at + 128 * 128, &tm_a, k * BK, m0, full(s));
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; s++) {
            tc::mbar_init(full(s), LOOSE ? 8 : 1);
            tc::mbar_init(empty(s), 1);
        }
        tc::mbar_init(done, 1);
        failed = 0;
        if (!LOOSE) {
            tc::prefetch_tensormap(&tm_w);
            tc::prefetch_tensormap(&tm_a);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no global read before this
    const int ahead = min(stages, k1 - k0);
    if (!LOOSE && threadIdx.x == 0)                        // the ring's first turn needs nothing but the barriers of this thread
        for (int i = 0; i < ahead; i++) load(k0 + i, i);
    if (warp == 1) tc::tmem_alloc<T::COLS>(tc::smem_addr(&tmem_at));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = tmem_at;

    if (warp == 0) {
        if (!LOOSE && lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            for (int k = k0 + ahead; k < k1; k++) {
                if (!wait(empty(s), phase)) { report(p); break; }
                load(k, s);
                if (++s == stages) { s = 0; phase ^= 1; }
            }
            for (int i = 0; i < ahead; i++) (void)wait(full(i), i < s ? phase ^ 1u : phase);   // none in flight
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t id = (1u << 4) | (p.dtype == KDA_BF16 ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(NT >> 3) << 17) | (8u << 24);
        int s = 0;
        uint32_t phase = 0;
        for (int k = k0; k < k1; k++) {
            if (!wait_warp(full(s), phase)) { report(p); failed = 1; break; }
            tc::fence_after_sync();
            const uint32_t at = s0 + s * T::STAGE;
            if (elect_one()) {
                mma_stage<1>(tmem, at, at + 128 * 128, id, k > k0);
                tc::commit(empty(s));
            }
            __syncwarp();
            if (++s == stages) { s = 0; phase ^= 1; }
        }
        if (elect_one()) tc::commit(done);
        __syncwarp();
    } else if (LOOSE && warp >= 2 + T::EW) {
        // lanes along the inner axis, two elements each; rows and columns past the matrices are zeros
        const uint16_t *pa = static_cast<const uint16_t *>(p.a), *pw = static_cast<const uint16_t *>(p.w);
        int s = 0;
        uint32_t phase = 1;
        for (int c = k0; c < k1; c++) {
            if (!wait_warp(empty(s), phase)) { report(p); break; }
            const int64_t k = static_cast<int64_t>(c) * BK + 2 * lane;
            unsigned char *at = sm + s * T::STAGE;
            static_assert((128 + NT) % 96 == 0 || !LOOSE, "");
#pragma unroll 1
            for (int r0 = warp - 2 - T::EW; r0 < 128 + NT; r0 += 96) {   // twelve rows' loads at once
                uint32_t x[12];
#pragma unroll
                for (int i = 0; i < 12; i++) {
                    const int r = r0 + 8 * i;
                    const int64_t row = r < 128 ? n0 + r : m0 + r - 128;
                    const uint16_t *from = r < 128 ? pw + row * p.ld_w : pa + row * p.ld_a;
                    const bool in = row < (r < 128 ? p.N : p.M);
                    const uint32_t lo = in && k < p.K ? from[k] : 0u, hi = in && k + 1 < p.K ? from[k + 1] : 0u;
                    x[i] = lo | hi << 16;
                }
#pragma unroll
                for (int i = 0; i < 12; i++) {
                    const int r = r0 + 8 * i;
                    *reinterpret_cast<uint32_t *>(at + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) = x[i];
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(full(s));
            if (++s == stages) { s = 0; phase ^= 1; }
        }
    }
    // the sums: a thread has one row of W, a column of the output
    const int quarter = warp % 4, n = n0 + quarter * 32 + lane;
    const bool epilogue = warp >= 2 && warp < 2 + T::EW;
    const int i0 = 16 * ((warp - 2) / 4), step = 16 * (T::EW / 4);          // rows of A in turn
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    if (epilogue && split == 1) {
        float r[16];
        fetch(p, r, m0 + i0, n);                           // beside the products
        bool ok = wait_warp(done, 0);
        tc::fence_after_sync();
        ok &= *static_cast<volatile uint32_t *>(&failed) == 0;
        if (!ok) report(p);
        for (int i = i0; ok && i < NT && m0 + i < p.M; i += step) {
            float v[16];
            tc::tmem_ld16(tq + i, v);
            tc::tmem_ld_wait();
            if (steps == 0) {
#pragma unroll
                for (int x = 0; x < 16; x++) v[x] = 0.f;
            }
            finish(p, v, r, m0 + i, n);
            if (i + step < NT) fetch(p, r, m0 + i + step, n);
        }
    }
    if (split > 1) {
        // every CTA's sums to its shared memory, then each joins its share of the rows of A
        float *sums = reinterpret_cast<float *>(sm);
        if (epilogue) {
            const bool ok = wait_warp(done, 0);
            tc::fence_after_sync();
            if (!ok) failed = 1;
#pragma unroll 1
            for (int i = i0; ok && i < NT && m0 + i < p.M; i += step) {
                float v[16];
                tc::tmem_ld16(tq + i, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 16; x++) sums[(i + x) * 132 + quarter * 32 + lane] = k1 > k0 ? v[x] : 0.f;
            }
        }
        __syncthreads();   // the copies' warp has seen all its copies land before the ring is taken for the sums: they are all the MMAs read
        cluster_sync();
        if (epilogue) {
            uint32_t bad = 0;
            for (int k = 0; k < split; k++) {
                uint32_t v;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cta(tc::smem_addr(&failed), k)));
                bad |= v;
            }
            if (bad) report(p);
            const int per = (NT / 16 + split - 1) / split * 16;
            for (int i = rank * per + i0; !bad && i < min(NT, (rank + 1) * per) && m0 + i < p.M; i += step) {
                float v[16] = {}, r[16];
                const int rows = min(16, p.M - m0 - i);
                fetch(p, r, m0 + i, n);
#pragma unroll 2
                for (int k = 0; k < split; k++) {
                    const uint32_t at = in_cta(tc::smem_addr(sums + i * 132 + quarter * 32 + lane), k);
                    float y[16];
#pragma unroll
                    for (int x = 0; x < 16; x++) {
                        y[x] = 0.f;
                        if (x < rows) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y[x]) : "r"(at + x * 132 * 4));
                    }
#pragma unroll
                    for (int x = 0; x < 16; x++) v[x] += y[x];
                }
                finish(p, v, r, m0 + i, n);
            }
        }
        cluster_sync();    // no CTA ends while another reads its sums
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) {
        (void)wait_warp(done, 0);
        tc::tmem_dealloc<T::COLS>(tmem);
    }
}

// ---- many rows: tiles of 256 x 256 by a pair of CTAs ----------------------------------------

struct Pair {
    static constexpr int EW = 8, THREADS = 128 + EW * 32;           // copies, MMAs, two idle warps, then the epilogue's: two for each quarter of the lanes
    static constexpr int STAGE = 2 * 128 * 128, STAGES = 5;         // per CTA: its 128 rows of A and its 128 rows of W
    static constexpr int BOX = 32 * 128;                            // 32 rows of 128 bytes of outputs, two for each epilogue warp
    static constexpr int BOXES = STAGES * STAGE, BARS = BOXES + EW * 2 * BOX, NBARS = 2 * STAGES + 4 + EW * 2, SMEM = BARS + NBARS * 8 + 16;
};
static_assert(Pair::SMEM <= 232448, "shared memory of a CTA");

struct Tiles {
    int m, n;          // tiles of 256
    int band;          // tiles of A that are walked together over all of W, so that W stays in L2
};
__device__ __forceinline__ void tile_at(const Tiles &t, int i, int *tm, int *tn)
{
    const int per = t.band * t.n, b = i / per, r = i % per, h = min(t.band, t.m - b * t.band);
    *tm = b * t.band + r % h;
    *tn = r / h;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_out,
            const __grid_constant__ CUtensorMap tm_res, const int tma_n, const __grid_constant__ MatmulParams p, const Tiles tiles)
{
    using T = Pair;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = tc::smem_addr(sm), b0 = s0 + T::BARS;
    volatile uint32_t *tmem_base = reinterpret_cast<uint32_t *>(sm + T::BARS + T::NBARS * 8);
    auto full = [&](int s) { return b0 + s * 8; };
    auto empty = [&](int s) { return b0 + (T::STAGES + s) * 8; };
    auto tfull = [&](int b) { return b0 + (2 * T::STAGES + b) * 8; };
    auto tempty = [&](int b) { return b0 + (2 * T::STAGES + 2 + b) * 8; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; s++) { tc::mbar_init(full(s), 1); tc::mbar_init(empty(s), 1); }
        for (int b = 0; b < 2; b++) { tc::mbar_init(tfull(b), 1); tc::mbar_init(tempty(b), 2 * T::EW); }
        for (int i = 0; i < T::EW * 2; i++) tc::mbar_init(b0 + (2 * T::STAGES + 4 + i) * 8, 1);
        tc::prefetch_tensormap(&tm_w);
        tc::prefetch_tensormap(&tm_a);
        if (tma_n > 0) tc::prefetch_tensormap(&tm_out);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no global read before this
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(b0 + T::NBARS * 8) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = *tmem_base;
    const int steps = (p.K + BK - 1) / BK, total = tiles.m * tiles.n, pairs = gridDim.x / 2, pair = blockIdx.x / 2;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int i = pair; i < total && ok; i += pairs) {
                int tm, tn;
                tile_at(tiles, i, &tm, &tn);
                const int m0 = tm * 256 + rank * 128, n0 = tn * 256 + rank * 128;
                for (int k = 0; k < steps; k++) {
                    if (!wait(empty(s), phase)) { report(p); ok = false; break; }
                    // both CTAs' copies are counted on the barrier of the one that issues the MMAs
                    if (rank == 0) tc::mbar_expect_tx(full(s), 2 * T::STAGE);
                    const uint32_t at = s0 + s * T::STAGE, bar = in_cta(full(s), 0);
                    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                                 " [%0], [%1, {%2, %3}], [%4];" :: "r"(at), "l"(&tm_a), "r"(k * BK), "r"(m0), "r"(bar) : "memory");
                    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                                 " [%0], [%1, {%2, %3}], [%4];" :: "r"(at + 128 * 128), "l"(&tm_w), "r"(k * BK), "r"(n0), "r"(bar) : "memory");
                    if (++s == T::STAGES) { s = 0; phase ^= 1; }
                }
            }
            // the last arrivals on this CTA's barriers come from the pair's other CTA: not before them does it end
            int k = s;
            uint32_t parity = phase;
            for (int i = 0; i < T::STAGES && ok; i++) {
                if (!wait(empty(k), parity)) { report(p); ok = false; }
                if (++k == T::STAGES) { k = 0; parity ^= 1; }
            }
            // where something gave up, both CTAs' copies: what was issued has long landed when this has run out
            if (!ok && rank == 0)
                for (int i = 0; i < T::STAGES; i++)
                    if (!wait(full(i), i < s ? phase ^ 1u : phase)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t id = (1u << 4) | (p.dtype == KDA_BF16 ? (1u << 7) | (1u << 10) : 0u) | (32u << 17) | (16u << 24);
            int s = 0, b = 0;
            uint32_t phase = 0, tphase = 1;
            bool ok = true;
            for (int i = pair; i < total && ok; i += pairs) {
                if (!wait_warp(tempty(b), tphase)) { report(p); break; }
                for (int k = 0; k < steps; k++) {
                    if (!wait_warp(full(s), phase)) { report(p); ok = false; break; }
                    tc::fence_after_sync();
                    const uint32_t at = s0 + s * T::STAGE;
                    if (elect_one()) {
                        mma_stage<2>(tmem + b * 256, at, at + 128 * 128, id, k > 0);
                        commit_pair(empty(s));
                        if (k == steps - 1) commit_pair(tfull(b));
                    }
                    __syncwarp();
                    if (++s == T::STAGES) { s = 0; phase ^= 1; }
                }
                if (ok && ++b == 2) { b = 0; tphase ^= 1; }
            }
            // no CTA ends with MMAs in flight: the last commit was on the stage before s
            (void)wait_warp(empty(s > 0 ? s - 1 : T::STAGES - 1), s > 0 ? phase : phase ^ 1u);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quarter = warp % 4, c0 = (warp - 4) / 4 * 128, e = warp - 4;   // TMEM lanes, columns of the tile
        const int es = p.out_dtype == KDA_FP32 ? 4 : 2, wide = 128 / es;         // columns of a box
        unsigned char *boxes = sm + T::BOXES + e * 2 * T::BOX;
        auto landed = [&](int x) { return b0 + (2 * T::STAGES + 4 + e * 2 + x) * 8; };
        uint32_t rphase = 0;                                                     // a bit for each box
        int b = 0, turn = 0;                                                     // boxes used so far: they take turns across tiles too
        uint32_t tphase = 0;
        for (int i = pair; i < total; i += pairs) {
            int tm, tn;
            tile_at(tiles, i, &tm, &tn);
            const int m0 = tm * 256 + rank * 128 + quarter * 32, n0 = tn * 256 + c0;
            const int blocks = m0 >= p.M || n0 >= p.N ? 0 : (min(128, p.N - n0) + wide - 1) / wide;   // of boxes that hold outputs
            auto side = [&](int x) { return (turn + x) & 1; };
            auto by_tma = [&](int x) { return n0 + (x + 1) * wide <= tma_n || (n0 + x * wide < tma_n && tma_n == p.N); };
            auto fetch = [&](int x) {                                             // the residual of box x
                if (lane == 0) {
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the box's last outputs are on their way
                    tc::mbar_expect_tx(landed(side(x)), T::BOX);
                    tc::tma_load_2d(tc::smem_addr(boxes + side(x) * T::BOX), &tm_res, n0 + x * wide, m0, landed(side(x)));
                }
                __syncwarp();
            };
            // box x between memory and shared memory where TMA cannot: row after row, lanes along the columns
            auto loose = [&](auto in, int x) {
                unsigned char *from = boxes + side(x) * T::BOX;
                const int cols = min(wide, p.N - n0 - x * wide), rows = min(32, p.M - m0);
#pragma unroll 4
                for (int r = 0; r < rows; r++) {
                    const int64_t at = static_cast<int64_t>(m0 + r) * (in ? p.ld_res : p.ld_out) + n0 + x * wide;
                    for (int c = lane; c < cols; c += 32) {
                        unsigned char *e = from + r * 128 + (((c * es >> 4) ^ (r & 7)) << 4) + (c * es & 15);
                        if (es == 4) {
                            if (in) *reinterpret_cast<uint32_t *>(e) = static_cast<const uint32_t *>(p.res)[at + c];
                            else static_cast<uint32_t *>(p.out)[at + c] = *reinterpret_cast<const uint32_t *>(e);
                        } else {
                            if (in) *reinterpret_cast<uint16_t *>(e) = static_cast<const uint16_t *>(p.res)[at + c];
                            else static_cast<uint16_t *>(p.out)[at + c] = *reinterpret_cast<const uint16_t *>(e);
                        }
                    }
                }
            };
            if (p.res && blocks > 0 && by_tma(0)) fetch(0);
            if (!wait_warp(tfull(b), tphase)) {
                report(p);
                if (p.res && blocks > 0 && by_tma(0)) (void)wait_warp(landed(side(0)), rphase >> side(0) & 1);   // no CTA ends with copies in flight
                break;
            }
            tc::fence_after_sync();
            const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * 256 + c0;
            bool gone = false;
#pragma unroll 1
            for (int x = 0; x < blocks; x++) {
                unsigned char *box = boxes + side(x) * T::BOX + lane * 128;
                const bool tma = by_tma(x);
                if (p.res && x + 1 < blocks && by_tma(x + 1)) fetch(x + 1);
                if (tma) {
                    if (p.res) {
                        if (!wait_warp(landed(side(x)), rphase >> side(x) & 1)) {
                            report(p);
                            if (x + 1 < blocks && by_tma(x + 1)) (void)wait_warp(landed(side(x + 1)), rphase >> side(x + 1) & 1);
                            gone = true;
                            break;
                        }
                        rphase ^= 1u << side(x);
                    } else {
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the last outputs but one: this box's
                        __syncwarp();
                    }
                } else {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
                    if (p.res) loose(std::true_type{}, x);
                    __syncwarp();
                }
#pragma unroll 1
                for (int h = 0; h < wide; h += 32) {
                    const int n = n0 + x * wide + h;
                    float v[32];
                    tmem_ld32(at + x * wide + h, v);
                    if (p.bias) {
                        const float own = n + lane < p.N ? load_as(p.bias, n + lane, p.bias_dtype) : 0.f;
#pragma unroll
                        for (int j = 0; j < 32; j++) v[j] += __shfl_sync(0xffffffffu, own, j);
                    }
                    activate(v, p.act);
                    // 16-byte piece j of the row is at j ^ (row % 8)
                    if (es == 4) {
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            float4 *to = reinterpret_cast<float4 *>(box + ((j ^ (lane & 7)) << 4));
                            float4 o = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                            if (p.res) { const float4 r = *to; o.x += r.x; o.y += r.y; o.z += r.z; o.w += r.w; }
                            *to = o;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            uint4 *to = reinterpret_cast<uint4 *>(box + (((h / 8 + j) ^ (lane & 7)) << 4));
                            uint32_t o[4];
                            if (p.res) {
                                const uint4 r = *to;
                                const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                                for (int q = 0; q < 4; q++) {
                                    float2 f;
                                    if (p.out_dtype == KDA_BF16) f = make_float2(__uint_as_float(rr[q] << 16), __uint_as_float(rr[q] & 0xffff0000u));
                                    else f = __half22float2(*reinterpret_cast<const __half2 *>(&rr[q]));
                                    v[8 * j + 2 * q] += f.x;
                                    v[8 * j + 2 * q + 1] += f.y;
                                }
                            }
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                o[q] = p.out_dtype == KDA_BF16 ? pack_bf16x2(v[8 * j + 2 * q], v[8 * j + 2 * q + 1]) : tc::pack_f16x2(v[8 * j + 2 * q], v[8 * j + 2 * q + 1]);
                            *to = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                if (tma) {
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                                     :: "l"(&tm_out), "r"(n0 + x * wide), "r"(m0), "r"(tc::smem_addr(boxes + side(x) * T::BOX)) : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    __syncwarp();
                } else {
                    __syncwarp();
                    loose(std::false_type{}, x);
                    tc::fence_proxy_async();   // the box may be TMA's next
                    __syncwarp();
                }
            }
            if (gone) break;
            turn += blocks;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(in_cta(tempty(b), 0)) : "memory");
            if (++b == 2) { b = 0; tphase ^= 1; }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc::fence_before_sync();
    cluster_sync();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

// ---- host ---------------------------------------------------------------------------------

// TMA's conditions; a single row has no pitch of its own.
bool tma_rows(const void *base, int64_t *ld, int64_t rows, int64_t cols, int es)
{
    const int per = 16 / es;
    if (rows == 1) *ld = (cols + per - 1) / per * per;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && *ld % per == 0 && *ld < (int64_t(1) << 37);
}

CUtensorMapDataType type_of(int dtype)
{
    return dtype == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : dtype == KDA_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
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

// What the launches need to know of a device, asked once and kept only on success: its multiprocessors, and how many CTAs of a
// kernel run at once in clusters of 1 .. 8 (clusters leave multiprocessors unused that do not fit their GPC).
struct Device {
    int sms = 0, fit[5][9] = {};   // tiles of 16, 32, 64 and 128 rows; loose ones

    template <int NT, bool LOOSE>
    cudaError_t ask_tile(int which)
    {
        using T = Tile<NT, LOOSE>;
        cudaError_t e = cudaFuncSetAttribute(tile_kernel<NT, LOOSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::ONE * T::STAGE);
        fit[which][1] = sms * (LOOSE ? 1 : 2);
        for (int split = 2; split <= 8 && e == cudaSuccess; split++) {
            Launch l(dim3(split), T::THREADS, T::TWO * T::STAGE, split, nullptr);
            l.at[0] = l.at[1];     // the cluster alone
            l.cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, tile_kernel<NT, LOOSE>, &l.cfg);
            fit[which][split] = n * split;
        }
        return e;
    }
    cudaError_t ask(int dev)
    {
        cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = ask_tile<16, false>(0);
        if (e == cudaSuccess) e = ask_tile<32, false>(1);
        if (e == cudaSuccess) e = ask_tile<64, false>(2);
        if (e == cudaSuccess) e = ask_tile<128, false>(3);
        if (e == cudaSuccess) e = ask_tile<64, true>(4);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pair::SMEM);
        return e;
    }
};

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

// How a call is computed.
struct Choice {
    int rows = 0;              // of A per tile: 16 .. 128 (tile_kernel), 256 (pair_kernel), 0: 64 loose ones
    int split = 1;
    int64_t ld_a, ld_w;
    bool boxes = false;        // the pairs' outputs, and residuals, move by TMA
    const Device *device = nullptr;
};

// Whether TMA can move the outputs, and the residual where there is one. (A plan without outputs takes them as such.)
bool outputs_by_tma(const MatmulParams &p)
{
    const int es = p.out_dtype == KDA_FP32 ? 4 : 2;
    int64_t ld_out = p.ld_out, ld_res = p.ld_res;
    return !p.out || (tma_rows(p.out, &ld_out, p.M, p.N, es) && (!p.res || tma_rows(p.res, &ld_res, p.M, p.N, es)));
}

// Plans are compared by their time in nanoseconds, fitted to the measured splits of products of 1 to 8192 rows, N and K of 64 to 12,288:
// start and end of a wave of CTAs, then its steps of 64 of the inner axis, each by the slowest of the MMAs, the stream from HBM (5.7 kB/ns
// over all multiprocessors) and the copies into a multiprocessor (107 B/ns), then the join of a split.
double time_tile(const MatmulParams &p, const int (&fit)[9], int nt, int split)
{
    if (fit[split] == 0) return 1e30;
    const int64_t tn = (p.N - 1) / 128 + 1, tm = (p.M - 1) / nt + 1, ctas = tn * tm * split;
    const int steps = (p.K + BK - 1) / BK;
    const double at_once = ctas < fit[split] ? ctas : fit[split], stage = (128 + nt) * 128.;
    const double hbm = at_once * 128 * 128 / tm / 5700., l2 = (at_once > fit[1] / 2 ? 2 : 1) * stage / 107.;
    double step = 264.;                                    // what one CTA's ring brings of W
    if (step < hbm) step = hbm;
    if (step < l2) step = l2;
    const double waves = static_cast<double>((ctas + fit[split] - 1) / fit[split]);
    return waves * (3200. + 14. * nt + step * ((steps + split - 1) / split)) + (split > 1 ? 1100. + 6. * nt : 0.);
}
// The pairs' epilogues are beside the next tile's MMAs. Where TMA cannot move outputs or residuals they go by rows through shared memory: a tile of
// 16-bit outputs then takes 7 to 9 us, of fp32 ones 11 to 20; with residuals 16 and 30 from L2, 48 and 90 from HBM, a row's latency after the other's.
double time_pair(const MatmulParams &p, int sms, bool boxes)
{
    const int64_t tiles = ((p.M - 1) / 256 + 1) * static_cast<int64_t>((p.N - 1) / 256 + 1);
    const int pairs = sms / 2, steps = (p.K + BK - 1) / BK;
    const double end = boxes ? 3000. : p.out_dtype == KDA_FP32 ? (p.res ? 90000. : 16000.) : (p.res ? 48000. : 9000.), main = 270. * steps;
    return 3000. + static_cast<double>((tiles + pairs - 1) / pairs) * (main > end ? main : end) + end;
}

cudaError_t choose(const MatmulParams &p, Choice *c)
{
    c->ld_a = p.ld_a;
    c->ld_w = p.ld_w;
    const cudaError_t e = this_device(&c->device);
    if (e != cudaSuccess) return e;
    const Device *d = c->device;
    double least = 1e30;
    auto tile = [&](int which, int nt, int as) {
        if ((static_cast<int64_t>(p.M) + nt - 1) / nt > 65535) return;       // the grid's y axis ends there
        for (int split = 1; split <= 8 && (split == 1 || split <= (p.K + BK - 1) / BK); split++) {
            const double t = time_tile(p, d->fit[which], nt, split);
            if (t < least) { least = t; c->rows = as; c->split = split; }
        }
    };
    if (p.K == 0 || !tma_rows(p.a, &c->ld_a, p.M, p.K, 2) || !tma_rows(p.w, &c->ld_w, p.N, p.K, 2)) {
        tile(4, 64, 0);
        return least < 1e30 ? cudaSuccess : cudaErrorInvalidConfiguration;
    }
    if (p.M <= 512) tile(0, 16, 16);
    if (p.M > 16 && p.M <= 1024) tile(1, 32, 32);
    if (p.M > 32) tile(2, 64, 64);
    if (p.M > 64) tile(3, 128, 128);
    c->boxes = outputs_by_tma(p);
    if (p.M > 128 && time_pair(p, d->sms, c->boxes) < least) { c->rows = 256; c->split = 1; }
    return cudaSuccess;
}

template <int NT, bool LOOSE>
cudaError_t run_tile(const MatmulParams &p, const Choice &c, cudaStream_t stream)
{
    using T = Tile<NT, LOOSE>;
    CUtensorMap ta = {}, tw = {};
    cudaError_t e;
    if (!LOOSE) {
        if ((e = encode(&tw, type_of(p.dtype), 2, p.w, p.K, p.N, c.ld_w, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
        if ((e = encode(&ta, type_of(p.dtype), 2, p.a, p.K, p.M, c.ld_a, BK, NT, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>((p.N - 1) / 128 + 1) * c.split, static_cast<unsigned>((p.M - 1) / NT + 1));
    // a CTA that has a multiprocessor to itself takes all of its shared memory: what is in flight is what its stream is bound by
    const int stages = static_cast<int64_t>(grid.x) * grid.y <= c.device->sms ? T::ONE : T::TWO;
    Launch l(grid, T::THREADS, stages * T::STAGE, c.split, stream);
    return cudaLaunchKernelEx(&l.cfg, tile_kernel<NT, LOOSE>, ta, tw, p, c.split, stages);
}

cudaError_t run_pair(const MatmulParams &p, const Choice &c, cudaStream_t stream)
{
    CUtensorMap ta, tw, to = {}, tr = {};
    cudaError_t e;
    if ((e = encode(&tw, type_of(p.dtype), 2, p.w, p.K, p.N, c.ld_w, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    if ((e = encode(&ta, type_of(p.dtype), 2, p.a, p.K, p.M, c.ld_a, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    const int es = p.out_dtype == KDA_FP32 ? 4 : 2, wide = 128 / es;
    // TMA writes whole 16-byte pieces, also where the map ends inside one: then the last columns are stored without it
    const int tma_n = !c.boxes ? 0 : static_cast<int64_t>(p.N) * es % 16 == 0 ? p.N : p.N / wide * wide;
    if (tma_n > 0 && (e = encode(&to, type_of(p.out_dtype), es, p.out, p.N, p.M, p.ld_out, wide, 32, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    if (tma_n > 0 && p.res && (e = encode(&tr, type_of(p.out_dtype), es, p.res, p.N, p.M, p.ld_res, wide, 32, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
        return e;
    const int sms = c.device->sms;
    const Tiles t{(p.M - 1) / 256 + 1, (p.N - 1) / 256 + 1, sms / 4};   // the pairs at work share two tiles of W
    const int64_t total = static_cast<int64_t>(t.m) * t.n;
    if (total > INT32_MAX - 4096) return cudaErrorInvalidConfiguration;
    const int pairs = static_cast<int>(total < sms / 2 ? total : sms / 2);
    return launch_pdl(pair_kernel, dim3(2 * pairs), dim3(Pair::THREADS), Pair::SMEM, stream, ta, tw, to, tr, tma_n, p, t);
}

}  // namespace

cudaError_t plan_matmul(const MatmulParams &p, int32_t (&plan)[2])
{
    Choice c;
    const cudaError_t e = choose(p, &c);
    plan[0] = c.rows;
    plan[1] = c.split;
    return e;
}

cudaError_t launch_matmul(const MatmulParams &p, cudaStream_t stream)
{
    Choice c;
    const cudaError_t e = choose(p, &c);
    if (e != cudaSuccess) return e;
    switch (c.rows) {
    case 16: return run_tile<16, false>(p, c, stream);
    case 32: return run_tile<32, false>(p, c, stream);
    case 64: return run_tile<64, false>(p, c, stream);
    case 128: return run_tile<128, false>(p, c, stream);
    case 256: return run_pair(p, c, stream);
    }
    return run_tile<64, true>(p, c, stream);
}

}  // namespace kda
