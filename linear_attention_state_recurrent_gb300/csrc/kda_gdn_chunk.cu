// The gated delta rule with one decay per head over packed sequences, in chunks of 64 rows on the tensor cores.
//
// With b the running log-decay inside a chunk, D[r, i] = e^{b_r - b_i}, A[r, i] = beta_r (k^_r . k^_i) D[r, i] for
// i < r and T = (I + A)^-1, a chunk is
//   Y = V - e^b (K^ S),   U = T diag(beta) Y,   O = e^b (Q^ S) + (Q^ K^^T * D, i <= r) U,   S <- e^{b_n} S + (K^ e^{b_n - b})^T U
// A decay that is the same in all channels leaves the tiles of q and k as they are in memory: every product takes them
// raw, as TMA brings them, and norms and decays are factors of rows and columns of the products. So nothing but T and the
// query-key products is computed ahead, and both beside the chain of chunks, in the same CTA: no workspace, one launch.
//
// One CTA per SM, persistent; it walks (sequence, value head) chains, longest sequences first. Its warps:
//   0 - 7    the chain: S in registers (fp32), transposed: a thread has one value column and half of the channels
//   8 - 15   two groups that take chunks in turn: decays, norms, T and the query-key products
//   16 - 19  outputs
//   20, 21   TMA; the chain's MMAs      22  the products K K^T and Q K^T
// The chain's products have value columns as rows (TMEM lanes), so that what depends on a token is a factor per column,
// and their first operand is written to TMEM by the thread that has the values.
// What enters the products is exact (q, k, v are bf16) or two bf16 terms, hi + lo = x to 2^-18.
#include <atomic>
#include <climits>
#include <mutex>
#include <type_traits>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_f32x2.cuh"
#include "kda_gdn_common.cuh"
#include "kda_pdl.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace gdn {
namespace {

constexpr int C = 64;                                  // rows of a chunk
constexpr int THREADS = 768;
constexpr int STAGES = 3;                              // chunks of q and k in shared memory (and two of v, which the chain reads first of all)
constexpr int SCALARS = 8;                             // chunks of row factors: the outputs may still read those of chunk c
                                                       // when those of c + 4 are written
constexpr int ORDER = 256;                             // sequences that are sorted by length
constexpr int BLK = 16 * 20;                           // floats of a 16 x 16 block, rows 20 apart: no bank conflicts
// registers: 80 a thread at launch, 61,440 in all; 256 x 136 + 256 x 64 + 2 x 128 x 40 = 61,440
constexpr int REG_CHAIN = 136, REG_PREP = 64, REG_OUT = 40, REG_REST = 40;

// columns of tensor memory
constexpr uint32_t T_S = 0;      // first operand of K S and Q S: the halves of the channels one after the other, each hi | lo; then the state's increment
constexpr uint32_t T_Y = 128;    // K S; then Y and later U (scaled), by halves of the rows, each hi | lo
constexpr uint32_t T_U = 192;    // U; then as an operand, by halves of the rows, each hi | lo
constexpr uint32_t T_O = 256;    // Q S and (Q K^T * D) U
constexpr uint32_t T_G = 384;    // K K^T | Q K^T, one for each of the two groups

struct Smem {
    static constexpr int HALF = 2 * C * 128;           // 64 channels of the chunk's keys, then of its queries
    static constexpr int STAGE = 2 * HALF, V = STAGES * STAGE, V_STAGE = C * 256;
    static constexpr int T = V + 2 * V_STAGE;          // per group T diag(beta), hi and lo, and the query-key products, hi and lo
    static constexpr int TILE = C * 128, GROUP = 4 * TILE;
    static constexpr int BLOCKS = T + 2 * GROUP;       // per group the ten blocks of A and T
    static constexpr int ROWS = BLOCKS + 2 * 10 * BLK * 4;
    static constexpr int SET = 3 * C + 4;              // floats: ys, us, qs, and gamma
    static constexpr int COLS = ROWS + SCALARS * SET * 4;   // per group: b hi, b lo, beta, and of the keys b lo less the norm's logarithm and e^{p - b} times the norm
    static constexpr int SORT = COLS + 2 * 5 * C * 4;
    static constexpr int BARS = SORT + ORDER * 2;
    static constexpr int NBARS = 2 * STAGES + 26;
    static constexpr int END = BARS + NBARS * 8 + 16;
};
static_assert(Smem::END <= 232448, "shared memory of a CTA");

struct Args {
    GdnParams p;
    const int32_t *cu;
    int rows, num_seqs;
};

// Matrix descriptors with the 128-byte swizzle, groups of 8 rows at 1024 bytes: the low words (the high one is the same for all).
// K-major: a row of the operand is 128 bytes.
__device__ __forceinline__ uint32_t desc_k(uint32_t at) { return (1u << 16) | (at >> 4); }
// The same bytes with the 128-byte rows along the inner axis (K^T from the tile of K): 64 columns, the next 64 at HALF.
__device__ __forceinline__ uint32_t desc_mn(uint32_t at) { return (static_cast<uint32_t>(Smem::HALF >> 4) << 16) | (at >> 4); }
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
// bf16 operands, fp32 sums, 128 rows; `mn`: the second operand is stored along its columns
constexpr uint32_t idesc(int n, bool mn = false)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// d (+)= a b^T, 16 of the inner axis; a in tensor memory
__device__ __forceinline__ void mma_t(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n"
                 :: "r"(d), "r"(a), "r"(b), "n"(DESC_HIGH), "r"(id), "r"(add ? 1u : 0u));
}
// The same with both operands from the same place in shared memory.
__device__ __forceinline__ void mma_gram(uint32_t d, uint32_t ab, uint32_t id, bool add)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%1, %2};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], db, db, %3, p;\n}\n"
                 :: "r"(d), "r"(ab), "n"(DESC_HIGH), "r"(id), "r"(add ? 1u : 0u));
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void arrive(uint32_t mbar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(mbar) : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N])
{
    static_assert(N == 16 || N == 32, "");
    if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                       "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                       "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                       "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                       "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                     : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
// d += a b in fp32 but for 2^-21 of the terms: tf32 products of the operands' two terms
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// The chunks of this CTA's chains, one after the other, the same for every warp.
struct Walk {
    const Args *a;
    const uint16_t *order;
    int item, total;            // chains: sequence (longest first) x value head
    int row, left, h;           // of the current chunk: its first row, the chain's rows from there on, the value head
    int seq;

    __device__ __forceinline__ Walk(const Args &args, const uint16_t *sorted)
        : a(&args), order(sorted), item(blockIdx.x), total(args.num_seqs * args.p.Hv) {}
    // CTA i's chains are i, 2 G - 1 - i, 2 G + i, ..: the longest with the shortest
    __device__ __forceinline__ void advance()
    {
        const int g = gridDim.x, at = item % g;
        item += 2 * (g - 1 - at) + 1;
    }
    // The chain at `item`: its rows, or none (an empty or bad range, a slot past the pool). *bad: error bits.
    __device__ __forceinline__ bool chain(uint32_t *bad = nullptr, int *all = nullptr)
    {
        const int s = item / a->p.Hv;
        h = item - s * a->p.Hv;
        seq = a->num_seqs <= ORDER ? order[s] : s;
        row = __ldg(a->cu + seq);
        const int end = __ldg(a->cu + seq + 1);
        left = end - row;
        uint32_t e = 0;
        if (row < 0 || end < row || end > a->rows) { left = 0; e |= kErrLengths; }
        if (all) *all = left;
        if (load_slot(a->p, seq) >= a->p.num_slots) { left = 0; e |= kErrSlotRange; }
        if (bad) *bad = e;
        return left > 0;
    }
    // To the first chunk at or after `item`; false: there is none.
    __device__ __forceinline__ bool begin()
    {
        while (item < total) {
            if (chain()) return true;
            advance();
        }
        return false;
    }
    __device__ __forceinline__ bool next()
    {
        row += C;
        left -= C;
        if (left > 0) return true;
        advance();
        return begin();
    }
    __device__ __forceinline__ int n() const { return left < C ? left : C; }
};

// A bounded wait that the CTA gives up as a whole: one that has run out (~2 s) says so to all the others.
struct Waiter {
    volatile uint32_t *gave_up;
    uint32_t *err;
    // Asleep for up to 1 ms a try: some twenty warps of a CTA wait at any time, and must not take the others' issue slots.
    __device__ __forceinline__ bool operator()(uint32_t mbar, uint32_t parity) const
    {
        long long start = 0;
        for (bool again = false;; again = true) {
            uint32_t ok;
            asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
                         " selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(mbar), "r"(parity), "r"(1000000u) : "memory");
            if (ok) return true;
            if (*gave_up) return false;
            const long long now = clock64();
            if (!again) start = now;
            else if (now - start > 4000000000ll) {
                *gave_up = 1;
                if (err) atomicOr(err, kErrTimeout);
                return false;
            }
        }
    }
    // by a converged warp, one answer for all lanes
    __device__ __forceinline__ bool warp(uint32_t mbar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, (*this)(mbar, parity));
    }
};

__device__ __forceinline__ constexpr int block_at(int a, int b) { return (a * (a + 1) / 2 + b) * BLK; }

template <int NH, int V>
__global__ void __launch_bounds__(THREADS, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tm_qk, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args a)
{
    constexpr int K = 64 * NH, KP = K / 2, VW = V / 32;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = tc::smem_addr(sm), b0 = s0 + Smem::BARS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // barriers
    auto full = [&](int s) { return b0 + s * 8; };                          // q and k of a chunk have landed
    auto empty = [&](int s) { return b0 + (STAGES + s) * 8; };              // and are no longer needed
    const uint32_t bx = b0 + 2 * STAGES * 8;
    const uint32_t s_ready = bx, ks_done = bx + 8, y_ready = bx + 16, u_ready = bx + 24, s_done = bx + 32, o_free = bx + 40;
    auto u_done = [&](int g) { return bx + 48 + g * 8; };
    auto o_done = [&](int g) { return bx + 64 + g * 8; };
    auto t_ready = [&](int g) { return bx + 80 + g * 8; };
    auto g_done = [&](int g) { return bx + 96 + g * 8; };
    auto g_free = [&](int g) { return bx + 112 + g * 8; };
    // a chunk's row factors are there: four of them, since those of c + 2 may be when the chain has yet to ask for those of c
    auto scaled = [&](uint32_t c) { return bx + 128 + (c & 3) * 8; };
    auto drained = [&](int i) { return bx + 160 + i * 8; };                 // the MMA warps' last commits
    auto v_full = [&](int i) { return bx + 176 + i * 8; };
    auto v_empty = [&](int i) { return bx + 192 + i * 8; };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(sm + Smem::BARS + Smem::NBARS * 8);   // tensor memory's base, whether a wait has given up
    uint16_t *order = reinterpret_cast<uint16_t *>(sm + Smem::SORT);
    float *sets = reinterpret_cast<float *>(sm + Smem::ROWS);
    const GdnParams &p = a.p;

    if (tid == 0) {
        for (int i = 0; i < STAGES; i++) { tc::mbar_init(full(i), 1); tc::mbar_init(empty(i), 1); }
        tc::mbar_init(s_ready, 2 * VW);
        tc::mbar_init(ks_done, 1);
        tc::mbar_init(y_ready, 2 * VW);
        tc::mbar_init(u_ready, 2 * VW);
        tc::mbar_init(s_done, 1);
        tc::mbar_init(o_free, VW);
        for (int g = 0; g < 2; g++) {
            tc::mbar_init(u_done(g), 1);
            tc::mbar_init(o_done(g), 1);
            tc::mbar_init(scaled(g), 4);
            tc::mbar_init(scaled(g + 2), 4);
            tc::mbar_init(drained(g), 1);
            tc::mbar_init(v_full(g), 1);
            tc::mbar_init(v_empty(g), 2 * VW);
            tc::mbar_init(t_ready(g), 4);
            tc::mbar_init(g_done(g), 1);
            tc::mbar_init(g_free(g), 4);
        }
        words[1] = 0;
        tc::prefetch_tensormap(&tm_qk);
        tc::prefetch_tensormap(&tm_v);
    }
    // above T's diagonal nothing is ever written
    for (int i = tid; i < 2 * Smem::GROUP / 16; i += THREADS) reinterpret_cast<uint4 *>(sm + Smem::T)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_proxy_async();
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no global read before this
    // the sequences by falling length: each finds its place
    if (a.num_seqs <= ORDER) {
        int *len = reinterpret_cast<int *>(sm);           // the first stage's place
        for (int i = tid; i < a.num_seqs; i += THREADS) len[i] = __ldg(a.cu + i + 1) - __ldg(a.cu + i);
        __syncthreads();
        for (int i = tid; i < a.num_seqs; i += THREADS) {
            const int own = len[i];
            int before = 0;
            for (int k = 0; k < a.num_seqs; k++) before += len[k] > own || (len[k] == own && k < i);
            order[before] = static_cast<uint16_t>(i);
        }
        tc::fence_proxy_async();                          // the place is TMA's from here on
    }
    if (warp == 21) tc::tmem_alloc<512>(s0 + Smem::BARS + Smem::NBARS * 8);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = words[0];
    const Waiter wait{words + 1, p.err};
    Walk w(a, order);

    if (warp < 8) {
        // ---- the chain ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REG_CHAIN));
        const int quarter = warp & 3, half = warp >> 2;
        if (quarter < VW) {
            const int j = quarter * 32 + lane;                                // this thread's value column
            const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t ts = t0 + T_S + half * KP, ty = t0 + T_Y + half * 32, tu = t0 + T_U + half * 32;
            float2 S[KP / 2];                                                 // channels KP half .. of column j
            auto give_s = [&] {                                               // S as the next products' operand
#pragma unroll
                for (int i = 0; i < KP / 2; i += 16) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int x = 0; x < 16; x++) split2(S[i + x].x, S[i + x].y, hi[x], lo[x]);
                    tmem_st16(ts + i, hi);
                    tmem_st16(ts + KP / 2 + i, lo);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(s_ready);
            };
            bool more = w.begin(), first = true;
            for (uint32_t c = 0; more; c++) {
                const int n = w.n();
                const uint32_t one = c & 1, two = (c >> 1) & 1;
                const int64_t slot = load_slot(p, w.seq);
                float *tile = slot >= 0 ? p.pool + slot * p.slot_stride + (static_cast<int64_t>(w.h) * K + half * KP) * V + j : nullptr;
                if (first) {
#pragma unroll
                    for (int i = 0; i < KP / 2; i++)
                        S[i] = slot >= 0 ? make_float2(tile[2 * i * V], tile[(2 * i + 1) * V]) : make_float2(0.f, 0.f);
                    give_s();
                }
                const bool last = w.left <= C;
                // v of this column, rows 32 half ..
                if (!wait.warp(v_full(c & 1), two)) break;
                uint32_t v[16];
                {
                    const unsigned char *at = sm + Smem::V + (c & 1) * Smem::V_STAGE + half * 32 * (V * 2) + j * 2;
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        v[i] = *reinterpret_cast<const uint16_t *>(at + 2 * i * V * 2) |
                               static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(at + (2 * i + 1) * V * 2)) << 16;
                }
                __syncwarp();
                if (lane == 0) arrive(v_empty(c & 1));
                if (!wait.warp(scaled(c), (c >> 2) & 1)) break;
                const float *set = sets + (c % SCALARS) * Smem::SET;
                const float gamma = set[3 * C];
                // Y = V - e^b K^ S; rows past the chunk's end are zeros, whatever is in memory there
                if (!wait.warp(ks_done, one)) break;
                tc::fence_after_sync();
                // (its terms go where later columns of K S still are: all of them first)
                {
                    uint32_t r[32];
                    tmem_ld(ty, r);
                    tc::tmem_ld_wait();
                    const float4 *ys = reinterpret_cast<const float4 *>(set + half * 32);
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int at = 8 * q + e;
                            const float4 f = ys[at / 2];
                            const float2 pk = make_float2(__uint_as_float(r[2 * at]), __uint_as_float(r[2 * at + 1]));
                            const float2 vv = make_float2(__uint_as_float(v[at] << 16), __uint_as_float(v[at] & 0xffff0000u));
                            float2 y = ffma2(at % 2 ? make_float2(-f.z, -f.w) : make_float2(-f.x, -f.y), pk, vv);
                            if (n < C) {
                                if (half * 32 + 2 * at >= n) y.x = 0.f;
                                if (half * 32 + 2 * at + 1 >= n) y.y = 0.f;
                            }
                            split2(y.x, y.y, hi[e], lo[e]);
                        }
                        tmem_st8(ty + 8 * q, hi);
                        tmem_st8(ty + 16 + 8 * q, lo);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(y_ready);
                // U: two terms for the outputs, two of its scaled form for the state
                if (!wait.warp(u_done(c & 1), two)) break;
                tc::fence_after_sync();
                {
                    uint32_t r[32];
                    tmem_ld(tu, r);
                    tc::tmem_ld_wait();
                    const float4 *us = reinterpret_cast<const float4 *>(set + C + half * 32);
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int at = 8 * q + e;
                            const float4 f = us[at / 2];
                            const float2 y = make_float2(__uint_as_float(r[2 * at]), __uint_as_float(r[2 * at + 1]));
                            const float2 z = fmul2(y, at % 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
                            split2(z.x, z.y, hi[e], lo[e]);
                        }
                        tmem_st8(ty + 8 * q, hi);
                        tmem_st8(ty + 16 + 8 * q, lo);
                    }
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            split2(__uint_as_float(r[2 * (8 * q + e)]), __uint_as_float(r[2 * (8 * q + e) + 1]), hi[e], lo[e]);
                        tmem_st8(tu + 8 * q, hi);
                        tmem_st8(tu + 16 + 8 * q, lo);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(u_ready);
                // S <- gamma S + its increment
                more = w.next();
                if (!wait.warp(s_done, one)) break;
                tc::fence_after_sync();
                const float2 g2 = make_float2(gamma, gamma);
#pragma unroll
                for (int i = 0; i < KP / 2; i += 16) {
                    uint32_t r[32];
                    tmem_ld(ts + 2 * i, r);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; x++) S[i + x] = ffma2(g2, S[i + x], make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])));
                }
                first = last;
                if (last) {
                    if (slot >= 0 && slot != p.null_slot) {
#pragma unroll
                        for (int i = 0; i < KP / 2; i++) {
                            tile[2 * i * V] = S[i].x;
                            tile[(2 * i + 1) * V] = S[i].y;
                        }
                    }
                } else {
                    give_s();
                }
            }
        }
    } else if (warp < 16) {
        // ---- T and the query-key products ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REG_PREP));
        const int g = (warp - 8) >> 2, t = tid & 127, pw = t >> 5, r = t & 63;   // thread t: row r of the keys (t < 64) or queries
        const bool query = t >= 64;
        unsigned char *tile = sm + Smem::T + g * Smem::GROUP;
        float *blocks = reinterpret_cast<float *>(sm + Smem::BLOCKS) + g * 10 * BLK;
        float *cols = reinterpret_cast<float *>(sm + Smem::COLS) + g * 5 * C;
        auto sync = [&] { asm volatile("bar.sync %0, 128;" :: "r"(1 + g) : "memory"); };
        // the same, with one answer to whether every thread's waits have come through
        auto sync_ok = [&](bool ok) {
            uint32_t all;
            asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.and.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
                         : "=r"(all) : "r"(1 + g), "r"(ok ? 1u : 0u) : "memory");
            return all != 0;
        };
        const int gq = lane >> 2, tq = lane & 3;
        // raw_g (warp 0) and raw_beta (warp 1) of rows 2 lane, 2 lane + 1 of the chunk at the walk
        float raw0 = 0.f, raw1 = 0.f, rate = 0.f, dtb = 0.f;
        int h_of = -1;
        auto fetch = [&] {
            if (pw < 2) {
                const uint16_t *at = pw == 0 ? p.rg : p.rb;
                const int64_t ld = pw == 0 ? p.ld_g : p.ld_beta, row = static_cast<int64_t>(w.row) + 2 * lane;
                const int n = w.n();
                if (2 * lane < n) raw0 = bf16_to_f32(__ldg(at + row * ld + w.h));
                if (2 * lane + 1 < n) raw1 = bf16_to_f32(__ldg(at + (row + 1) * ld + w.h));
            }
        };
        bool more = w.begin();
        if (more && g == 1) more = w.next();
        if (more) fetch();
        for (uint32_t c = g; more; c += 2) {
            const int s = c % STAGES, n = w.n(), h = w.h;
            const uint32_t two = (c >> 1) & 1;
            const float in0 = raw0, in1 = raw1;
            more = w.next() && w.next();                                     // this group's next chunk
            if (more) fetch();
            float *set = sets + (c % SCALARS) * Smem::SET;
            if (pw == 0) {                                                    // the running decay, in units of log 2
                if (h != h_of) {
                    h_of = h;
                    rate = expf(__ldg(p.A_log + h)) * -1.44269504f;
                    dtb = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
                }
                const double g0 = 2 * lane < n ? rate * softplus_f(in0 + dtb) : 0.f, g1 = 2 * lane + 1 < n ? rate * softplus_f(in1 + dtb) : 0.f;
                double b = g0 + g1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double x = __shfl_up_sync(0xffffffffu, b, o);
                    if (lane >= o) b += x;
                }
                const double b0_ = b - g1;
                const float h0 = static_cast<float>(b0_), h1 = static_cast<float>(b);
                *reinterpret_cast<float2 *>(cols + 2 * lane) = make_float2(h0, h1);
                *reinterpret_cast<float2 *>(cols + C + 2 * lane) = make_float2(static_cast<float>(b0_ - h0), static_cast<float>(b - h1));
            } else if (pw == 1) {
                *reinterpret_cast<float2 *>(cols + 2 * C + 2 * lane) =
                    make_float2(2 * lane < n ? sigmoid_f(in0) : 0.f, 2 * lane + 1 < n ? sigmoid_f(in1) : 0.f);
            }
            // the norm of this thread's row
            bool ok = wait.warp(full(s), (c / STAGES) & 1);
            float2 sum = make_float2(0.f, 0.f);
            unsigned char *own = sm + s * Smem::STAGE + t * 128;
#pragma unroll
            for (int hf = 0; hf < NH; hf++)
#pragma unroll
                for (int x = 0; x < 8; x++) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(own + hf * Smem::HALF + ((x ^ (t & 7)) << 4));
                    const uint32_t qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        const float2 f = make_float2(__uint_as_float(qq[y] << 16), __uint_as_float(qq[y] & 0xffff0000u));
                        sum = ffma2(f, f, sum);
                    }
                }
            const float norm = r < n ? rsqrtf(sum.x + sum.y + p.eps) : 0.f;
            if (!query && r >= n) {   // keys of other sequences: 0 times what they may hold is not 0
#pragma unroll
                for (int hf = 0; hf < NH; hf++)
#pragma unroll
                    for (int x = 0; x < 8; x++) *reinterpret_cast<uint4 *>(own + hf * Smem::HALF + (x << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (!sync_ok(ok)) break;
            const float b_hi = cols[r], b_lo = cols[C + r];
            const float scale = (query ? p.scale : cols[2 * C + r]) * norm;
            if (!query) {
                const float e_hi = cols[C - 1], e_lo = cols[2 * C - 1];
                set[r] = ex2(b_hi + b_lo) * norm;
                set[C + r] = ex2((e_hi - b_hi) + (e_lo - b_lo)) * norm;
                if (r == 0) set[3 * C] = ex2(e_hi + e_lo);
                cols[3 * C + r] = b_lo - (r < n ? __log2f(norm) : 0.f);
                cols[4 * C + r] = ex2((cols[r | 15] - b_hi) + (cols[C + (r | 15)] - b_lo)) * norm;
            } else {
                set[2 * C + r] = p.scale * ex2(b_hi + b_lo) * norm;
            }
            __syncwarp();
            if (lane == 0) arrive(scaled(c));
            sync();
            // K K^T and Q K^T: row r of A (its blocks up to the diagonal's), or of the query-key products
            ok = wait.warp(g_done(g), two);
            tc::fence_after_sync();
            if (query && c >= 2) ok &= wait.warp(o_done(g), two ^ 1);         // the products of this group's last chunk have been used
            const int low = (pw & 1) * 2;                                     // the first block with a diagonal in the warp's rows
            const uint32_t tg = tmem + T_G + g * 64 + (static_cast<uint32_t>(pw * 32) << 16);
            float2 d[8];
            auto put = [&](int bl) {
                if (query) {
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) split2(d[4 * y + i].x, d[4 * y + i].y, hi[i], lo[i]);
                        unsigned char *at = tile + 2 * Smem::TILE + r * 128 + (((2 * bl + y) ^ (r & 7)) << 4);
                        *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(at + Smem::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                } else if (bl <= r >> 4) {
                    float *at = blocks + block_at(r >> 4, bl) + (r & 15) * 20;
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        *reinterpret_cast<float4 *>(at + 4 * i) = make_float4(d[2 * i].x, d[2 * i].y, d[2 * i + 1].x, d[2 * i + 1].y);
                }
            };
            // blocks left of it: e^{b_r - b_i} = e^{b_r - p} e^{p - b_i}, p the sum at the block's last row: neither is above 1
#pragma unroll 1
            for (int bl = 0; bl < low; bl++) {
                uint32_t x[16];
                tmem_ld(tg + bl * 16, x);
                const float f = ex2((b_hi - cols[bl * 16 + 15]) + (b_lo - cols[C + bl * 16 + 15])) * scale;
                const float2 f2 = make_float2(f, f);
                tc::tmem_ld_wait();
                if (r >= n) {                                                 // not a row of the chunk: whatever it held
#pragma unroll
                    for (int i = 0; i < 16; i++) x[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 e = *reinterpret_cast<const float4 *>(cols + 4 * C + bl * 16 + 4 * i);
                    d[2 * i] = fmul2(fmul2(make_float2(e.x, e.y), f2), make_float2(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])));
                    d[2 * i + 1] = fmul2(fmul2(make_float2(e.z, e.w), f2), make_float2(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])));
                }
                put(bl);
            }
            // and the two with diagonals: entry by entry, the ones above it cut off
            const int end = r < n ? r + query : 0;
            const float2 bh = make_float2(b_hi, b_hi), bl2 = make_float2(b_lo, b_lo), sc = make_float2(scale, scale);
#pragma unroll 1
            for (int bl = low; bl < low + 2; bl++) {
                uint32_t x[16];
                tmem_ld(tg + bl * 16, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 eh = *reinterpret_cast<const float4 *>(cols + bl * 16 + 4 * i);
                    const float4 el = *reinterpret_cast<const float4 *>(cols + 3 * C + bl * 16 + 4 * i);
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const float2 e = fadd2(fsub2(bh, y ? make_float2(eh.z, eh.w) : make_float2(eh.x, eh.y)),
                                               fsub2(bl2, y ? make_float2(el.z, el.w) : make_float2(el.x, el.y)));
                        const float2 v = fmul2(fmul2(make_float2(ex2(e.x), ex2(e.y)), sc),
                                               make_float2(__uint_as_float(x[4 * i + 2 * y]), __uint_as_float(x[4 * i + 2 * y + 1])));
                        const int col = bl * 16 + 4 * i + 2 * y;
                        d[2 * i + y] = make_float2(col < end ? v.x : 0.f, col + 1 < end ? v.y : 0.f);
                    }
                }
                put(bl);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(g_free(g));
            sync();
            // T: the diagonal blocks, a warp each, by substitution; a lane has a column (lanes 16 and up the same again)
            {
                const float *A = blocks + block_at(pw, pw);
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    float y[4] = {i == (lane & 15) ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < i; k += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(A + i * 20 + k);
                        y[0] = fmaf(-f.x, x[k], y[0]);
                        if (k + 1 < i) y[1] = fmaf(-f.y, x[k + 1], y[1]);
                        if (k + 2 < i) y[2] = fmaf(-f.z, x[k + 2], y[2]);
                        if (k + 3 < i) y[3] = fmaf(-f.w, x[k + 3], y[3]);
                    }
                    x[i] = (y[0] + y[1]) + (y[2] + y[3]);
                }
                __syncwarp();
                if (lane < 16)
#pragma unroll
                    for (int i = 0; i < 16; i++) blocks[block_at(pw, pw) + i * 20 + lane] = x[i];
            }
            sync();
            // the blocks below them: [[X, 0], [-Y A X, Y]], first of 32 rows, then of all 64. X^T A^T is the first operand of the
            // second product as it leaves the first one: column 2t of a tile counts as k = t, 2t + 1 as k = t + 4.
            {
                const int pr = pw >> 1, hf = pw & 1;
                const float *X = blocks + block_at(2 * pr, 2 * pr), *Y = blocks + block_at(2 * pr + 1, 2 * pr + 1);
                float *A = blocks + block_at(2 * pr + 1, 2 * pr);
                float xa[2][4] = {}, out[4] = {};
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    Tf32<4> fx;
                    fx.set(0, X[(8 * k + tq) * 20 + gq]);
                    fx.set(1, X[(8 * k + tq) * 20 + gq + 8]);
                    fx.set(2, X[(8 * k + tq + 4) * 20 + gq]);
                    fx.set(3, X[(8 * k + tq + 4) * 20 + gq + 8]);
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        Tf32<2> fa;
                        fa.set(0, A[(8 * m + gq) * 20 + 8 * k + tq]);
                        fa.set(1, A[(8 * m + gq) * 20 + 8 * k + tq + 4]);
                        mma_split(xa[m], fx, fa);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    Tf32<4> fx;
                    Tf32<2> fy;
                    fx.set(0, -xa[m][0]); fx.set(1, -xa[m][2]); fx.set(2, -xa[m][1]); fx.set(3, -xa[m][3]);
                    const float2 y = *reinterpret_cast<const float2 *>(Y + (8 * hf + gq) * 20 + 8 * m + 2 * tq);
                    fy.set(0, y.x);
                    fy.set(1, y.y);
                    mma_split(out, fx, fy);
                }
                sync();                                                       // A has been read
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const int col = gq + 8 * (x >> 1), row = 8 * hf + 2 * tq + (x & 1);
                    A[row * 20 + col] = out[x];
                }
            }
            sync();
            {
                const int mt = pw >> 1, hf = pw & 1;                          // columns 16 mt .., rows 32 + 16 hf ..
                float out[2][4] = {};
#pragma unroll
                for (int ib = 0; ib < 2; ib++) {
                    if (ib > hf) break;
                    float xa[2][4] = {};
#pragma unroll
                    for (int kb = 0; kb < 2; kb++) {
                        if (kb < mt) continue;
                        const float *X = blocks + block_at(kb, mt), *A = blocks + block_at(2 + ib, kb);
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            Tf32<4> fx;
                            fx.set(0, X[(8 * k + tq) * 20 + gq]);
                            fx.set(1, X[(8 * k + tq) * 20 + gq + 8]);
                            fx.set(2, X[(8 * k + tq + 4) * 20 + gq]);
                            fx.set(3, X[(8 * k + tq + 4) * 20 + gq + 8]);
#pragma unroll
                            for (int m = 0; m < 2; m++) {
                                Tf32<2> fa;
                                fa.set(0, A[(8 * m + gq) * 20 + 8 * k + tq]);
                                fa.set(1, A[(8 * m + gq) * 20 + 8 * k + tq + 4]);
                                mma_split(xa[m], fx, fa);
                            }
                        }
                    }
                    const float *Y = blocks + block_at(2 + hf, 2 + ib);
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        Tf32<4> fx;
                        fx.set(0, -xa[m][0]); fx.set(1, -xa[m][2]); fx.set(2, -xa[m][1]); fx.set(3, -xa[m][3]);
#pragma unroll
                        for (int rt = 0; rt < 2; rt++) {
                            Tf32<2> fy;
                            const float2 y = *reinterpret_cast<const float2 *>(Y + (8 * rt + gq) * 20 + 8 * m + 2 * tq);
                            fy.set(0, y.x);
                            fy.set(1, y.y);
                            mma_split(out[rt], fx, fy);
                        }
                    }
                }
                sync();                                                       // A has been read
                float *at = blocks + block_at(2 + hf, mt);
#pragma unroll
                for (int rt = 0; rt < 2; rt++)
#pragma unroll
                    for (int x = 0; x < 4; x++) at[(8 * rt + 2 * tq + (x & 1)) * 20 + gq + 8 * (x >> 1)] = out[rt][x];
            }
            if (c >= 2) ok &= wait.warp(u_done(g), two ^ 1);                  // T of this group's last chunk has been used
            if (!sync_ok(ok)) break;
            // T diag(beta), hi and lo: half of row r
#pragma unroll 1
            for (int bl = t >> 6 << 1; bl <= r >> 4 && bl < (t >> 6 << 1) + 2; bl++) {
                const float *from = blocks + block_at(r >> 4, bl) + (r & 15) * 20;
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float4 x = *reinterpret_cast<const float4 *>(from + 8 * y + 4 * i);
                        const float4 e = *reinterpret_cast<const float4 *>(cols + 2 * C + bl * 16 + 8 * y + 4 * i);
                        const float2 v0 = fmul2(make_float2(x.x, x.y), make_float2(e.x, e.y)), v1 = fmul2(make_float2(x.z, x.w), make_float2(e.z, e.w));
                        split2(v0.x, v0.y, hi[2 * i], lo[2 * i]);
                        split2(v1.x, v1.y, hi[2 * i + 1], lo[2 * i + 1]);
                    }
                    unsigned char *at = tile + r * 128 + (((2 * bl + y) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + Smem::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(t_ready(g));
            sync();                                                           // blocks and columns are free again
        }
    } else if (warp < 20) {
        // ---- outputs ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REG_OUT));
        const int quarter = warp & 3, j = quarter * 32 + lane;
        // chains that are skipped: their error bits, and zeros for a slot past the pool
        for (Walk z(a, order); z.item < z.total; z.advance()) {
            uint32_t bad;
            int all;
            z.chain(&bad, &all);
            if (!bad) continue;
            if (p.err && quarter == 0 && lane == 0) atomicOr(p.err, bad);
            if (j < V)
                for (int i = 0; i < all; i++) p.out[(static_cast<int64_t>(z.row) + i) * p.ld_out + static_cast<int64_t>(z.h) * V + j] = 0;
        }
        if (quarter < VW) {
            const uint32_t t0 = tmem + T_O + (static_cast<uint32_t>(quarter * 32) << 16);
            bool more = w.begin();
            for (uint32_t c = 0; more; c++) {
                const int n = w.n();
                uint16_t *out = p.out + static_cast<int64_t>(w.row) * p.ld_out + static_cast<int64_t>(w.h) * V + j;
                const float *qs = sets + (c % SCALARS) * Smem::SET + 2 * C;
                if (!wait.warp(o_done(c & 1), (c >> 1) & 1)) break;
                tc::fence_after_sync();
                more = w.next();
                auto store = [&](auto whole) {
#pragma unroll
                    for (int i = 0; i < C; i += 8) {
                        uint32_t x[8], y[8];
                        tmem_ld8(t0 + i, x);
                        tmem_ld8(t0 + C + i, y);
                        tc::tmem_ld_wait();
                        if (i == C - 8) {
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) arrive(o_free);
                        }
#pragma unroll
                        for (int r = 0; r < 8; r += 2) {
                            const float2 o = ffma2(*reinterpret_cast<const float2 *>(qs + i + r), make_float2(__uint_as_float(x[r]), __uint_as_float(x[r + 1])),
                                                   make_float2(__uint_as_float(y[r]), __uint_as_float(y[r + 1])));
                            const uint32_t o2 = pack_bf16x2(o.x, o.y);
                            if (whole || i + r < n) *out = static_cast<uint16_t>(o2);
                            out += p.ld_out;
                            if (whole || i + r + 1 < n) *out = static_cast<uint16_t>(o2 >> 16);
                            out += p.ld_out;
                        }
                    }
                };
                if (n == C) store(std::true_type{});
                else store(std::false_type{});
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REG_REST));
        if (warp == 20) {
            // ---- TMA ----
            if (lane == 0) {
                const int hk = p.Hv / p.Hk;
                bool more = w.begin();
                uint32_t c = 0;
                for (; more; c++) {
                    const int s = c % STAGES;
                    if (c >= STAGES && !wait(empty(s), (c / STAGES - 1) & 1)) break;
                    const uint32_t at = s0 + s * Smem::STAGE;
                    tc::mbar_expect_tx(full(s), NH * Smem::HALF);
#pragma unroll
                    for (int hf = 0; hf < NH; hf++) {
                        const int x = w.h / hk * K + 64 * hf;
                        tc::tma_load_2d(at + hf * Smem::HALF, &tm_qk, p.Hk * K + x, w.row, full(s));
                        tc::tma_load_2d(at + hf * Smem::HALF + C * 128, &tm_qk, x, w.row, full(s));
                    }
                    if (c >= 2 && !wait(v_empty(c & 1), ((c >> 1) & 1) ^ 1)) {
                        (void)tc::mbar_wait(full(s), (c / STAGES) & 1);
                        break;
                    }
                    tc::mbar_expect_tx(v_full(c & 1), C * V * 2);
                    tc::tma_load_2d(s0 + Smem::V + (c & 1) * Smem::V_STAGE, &tm_v, 2 * p.Hk * K + w.h * V, w.row, v_full(c & 1));
                    more = w.next();
                }
                // no CTA ends with copies in flight
                for (uint32_t k = c > STAGES ? c - STAGES : 0; k < c; k++) (void)tc::mbar_wait(full(k % STAGES), (k / STAGES) & 1);
                for (uint32_t k = c > 2 ? c - 2 : 0; k < c; k++) (void)tc::mbar_wait(v_full(k & 1), (k >> 1) & 1);
            }
        } else if (warp == 21) {
            // ---- the chain's MMAs ----
            bool more = w.begin();
            for (uint32_t c = 0; more; c++) {
                const int s = c % STAGES, g = c & 1;
                const uint32_t one = c & 1, two = (c >> 1) & 1;
                const uint32_t at = s0 + s * Smem::STAGE, tt = s0 + Smem::T + g * Smem::GROUP;
                if (!wait.warp(full(s), (c / STAGES) & 1) || !wait.warp(s_ready, one)) break;
                tc::fence_after_sync();
                if (elect_one()) {
                    // K S, both terms of S
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int k = 0; k < K / 16; k++) {
                            const int half = k / (KP / 16), kk = k % (KP / 16);
                            mma_t(tmem + T_Y, tmem + T_S + half * KP + x * (KP / 2) + kk * 8, desc_k(at + (k / 4) * Smem::HALF + (k % 4) * 32), idesc(C), x + k > 0);
                        }
                    tc::commit(ks_done);
                }
                __syncwarp();
                if (c > 0 && !wait.warp(o_free, one ^ 1)) break;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int k = 0; k < K / 16; k++) {
                            const int half = k / (KP / 16), kk = k % (KP / 16);
                            mma_t(tmem + T_O, tmem + T_S + half * KP + x * (KP / 2) + kk * 8, desc_k(at + (k / 4) * Smem::HALF + C * 128 + (k % 4) * 32), idesc(C), x + k > 0);
                        }
                }
                __syncwarp();
                if (!wait.warp(t_ready(g), two) || !wait.warp(y_ready, one)) break;
                tc::fence_after_sync();
                if (elect_one()) {
                    // U = (T diag(beta)) Y: hi hi, lo hi, hi lo. Rows of T before 16 k are zero in columns 16 k ..
#pragma unroll
                    for (int x = 0; x < 3; x++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_t(tmem + T_U + 16 * k, tmem + T_Y + (k / 2) * 32 + (x == 1 ? 16 : 0) + (k % 2) * 8,
                                  desc_k(tt + (x == 2 ? Smem::TILE : 0) + 16 * k * 128 + k * 32), idesc(C - 16 * k), x + k > 0);
                    tc::commit(u_done(g));
                }
                __syncwarp();
                if (!wait.warp(u_ready, one)) break;
                tc::fence_after_sync();
                if (elect_one()) {
                    // the state's increment, both terms of U
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_t(tmem + T_S, tmem + T_Y + (k / 2) * 32 + x * 16 + (k % 2) * 8, desc_mn(at + k * 16 * 128), idesc(K, true), x + k > 0);
                    tc::commit(s_done);
#pragma unroll
                    for (int x = 0; x < 3; x++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_t(tmem + T_O + C + 16 * k, tmem + T_U + (k / 2) * 32 + (x == 1 ? 16 : 0) + (k % 2) * 8,
                                  desc_k(tt + (x == 2 ? 3 : 2) * Smem::TILE + 16 * k * 128 + k * 32), idesc(C - 16 * k), x + k > 0);
                    tc::commit(empty(s));
                    tc::commit(o_done(g));
                }
                __syncwarp();
                more = w.next();
            }
            // nor with MMAs
            if (elect_one()) tc::commit(drained(0));
            __syncwarp();
            (void)tc::mbar_wait(drained(0), 0);
        } else if (warp == 22) {
            // ---- K K^T and Q K^T ----
            bool more = w.begin();
            for (uint32_t c = 0; more; c++) {
                const int s = c % STAGES, g = c & 1;
                const uint32_t at = s0 + s * Smem::STAGE;
                if (!wait.warp(full(s), (c / STAGES) & 1)) break;
                if (c >= 2 && !wait.warp(g_free(g), ((c >> 1) & 1) ^ 1)) break;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < K / 16; k++)
                        mma_gram(tmem + T_G + g * 64, desc_k(at + (k / 4) * Smem::HALF + (k % 4) * 32), idesc(C), k > 0);
                    tc::commit(g_done(g));
                }
                __syncwarp();
                more = w.next();
            }
            if (elect_one()) tc::commit(drained(1));
            __syncwarp();
            (void)tc::mbar_wait(drained(1), 0);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 21) tc::tmem_dealloc<512>(tmem);
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

// Boxes of 64 rows by `box` columns of the packed q | k | v rows.
cudaError_t encode(CUtensorMap *m, const GdnParams &p, int64_t rows, int64_t cols, int box, CUtensorMapSwizzle swizzle)
{
    const auto enc = encoder();
    if (!enc) return cudaErrorSymbolNotFound;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.ld_qkv) * 2};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), C}, steps[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(p.qkv), dims, strides, boxes, steps,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The multiprocessors of the current device, the kernels' shared-memory limits set there, once; kept only on success.
cudaError_t this_device(int *sms)
{
    constexpr int MOST = 64;
    static int counts[MOST];
    static std::atomic<bool> known[MOST];
    static std::mutex asking;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= MOST) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        const std::lock_guard<std::mutex> one(asking);
        if (!known[dev].load(std::memory_order_relaxed)) {
            const auto limit = [&](auto kernel) {
                if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::END);
            };
            e = cudaDeviceGetAttribute(&counts[dev], cudaDevAttrMultiProcessorCount, dev);
            limit(chunk_kernel<1, 32>); limit(chunk_kernel<1, 64>); limit(chunk_kernel<1, 128>);
            limit(chunk_kernel<2, 32>); limit(chunk_kernel<2, 64>); limit(chunk_kernel<2, 128>);
            if (e != cudaSuccess) return e;
            known[dev].store(true, std::memory_order_release);
        }
    }
    *sms = counts[dev];
    return cudaSuccess;
}

}  // namespace
}  // namespace gdn

cudaError_t launch_gdn_prefill(const GdnParams &p, int K, int V, const int32_t *cu, int64_t rows, int64_t num_seqs,
                               cudaStream_t stream)
{
    using namespace gdn;
    // TMA wants rows on 16-byte boundaries, and tiles of 64 channels: the rest goes in blocks of 16 rows
    if (K == 32 || reinterpret_cast<uintptr_t>(p.qkv) % 16 != 0 || p.ld_qkv % 8 != 0 || p.ld_qkv >= (int64_t(1) << 38))
        return launch_gdn_rows(p, K, V, 16, cu, rows, num_seqs, stream);
    int sms;
    cudaError_t e = this_device(&sms);
    if (e != cudaSuccess) return e;
    CUtensorMap qk, v;
    const int64_t cols = 2 * static_cast<int64_t>(p.Hk) * K + static_cast<int64_t>(p.Hv) * V;
    if ((e = encode(&qk, p, rows, cols, 64, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    if ((e = encode(&v, p, rows, cols, V, CU_TENSOR_MAP_SWIZZLE_NONE)) != cudaSuccess) return e;
    const Args a{p, cu, static_cast<int>(rows), static_cast<int>(num_seqs)};
    const int64_t chains = num_seqs * p.Hv;
    const dim3 grid(static_cast<unsigned>(chains < sms ? chains : sms));
#define KDA_GDN_RUN(NH, VV) \
    if (K == 64 * NH && V == VV) return launch_pdl(chunk_kernel<NH, VV>, grid, dim3(THREADS), Smem::END, stream, qk, v, a);
    KDA_GDN_RUN(1, 32) KDA_GDN_RUN(1, 64) KDA_GDN_RUN(1, 128) KDA_GDN_RUN(2, 32) KDA_GDN_RUN(2, 64) KDA_GDN_RUN(2, 128)
#undef KDA_GDN_RUN
    return cudaErrorInvalidValue;
}

}  // namespace kda
