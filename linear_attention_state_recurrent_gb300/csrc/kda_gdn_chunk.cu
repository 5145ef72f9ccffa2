// The gated delta rule with one decay per head over packed sequences, in chunks of 64 rows on the tensor cores.
//
// With b the running log-decay inside a chunk, D[r, i] = e^{b_r - b_i}, A[r, i] = (k^_r . k^_i) D[r, i] beta_i for
// i < r and T = (I + A)^-1, a chunk is
//   Y = V - e^b (K^ S),   Z = T Y,   O = e^b (Q^ S) + W Z,  W = (Q^ K^^T * D) diag(beta) (i <= r),   S <- e^{b_n} S + (K^ e^{b_n - b} beta)^T Z
// (beta stands behind T, whose diagonal is then one: Y goes into Z's sums as it is, in fp32, and through products only what is off the diagonal.)
// A decay that is the same in all channels leaves the tiles of q and k as they are in memory: every product takes them
// raw, as TMA brings them, and norms and decays are factors of rows and columns of the products. What the chunks need but for
// S, T and W, is 21 KB a chunk and head (KDA's is 58 KB). Three launches, and two more
// where few long sequences are cut into parts that go side by side:
//   map_kernel    where each sequence's chunks are, from cu_seqlens on the device
//   prep_kernel   T, W and the row factors of every chunk at once: a CTA per chunk and key head, for all its value heads
//   chain_kernel  one CTA per SM walks (sequence, value head) chains, longest sequences first, S in registers
//   ends_kernel, outputs_kernel   join the parts
// The chain's products have value columns as rows (TMEM lanes), so that what depends on a token is a factor per column,
// and their first operand is written to TMEM by the thread that has the values.
// What enters the products is exact (q, k, v are bf16), two bf16 terms, hi + lo = x to 2^-17, or, of Z on its way into the state, three (2^-25).
#include <atomic>
#include <climits>
#include <mutex>
#include <type_traits>

#include "kda_f32x2.cuh"
#include "kda_gdn_common.cuh"
#include "kda_mma.cuh"
#include "kda_pdl.cuh"

namespace kda {
namespace gdn {
namespace {

using mma::arrive;
using mma::elect_one;
using mma::phase_over;

constexpr int C = 64;                                  // rows of a chunk
constexpr int ORDER = 256;                             // sequences that are sorted by length
constexpr int BLK = 16 * 20;                           // floats of a 16 x 16 block, rows 20 apart: no bank conflicts

// A chunk and head's record. Of the 64 x 64 matrices T - I and W, hi and lo each, the blocks on and below the diagonal: a panel
// for every 16 columns with the rows from 16 k on, in the order the MMAs read without a swizzle (8 rows of 16 bytes follow each
// other, the next 8 columns 128 bytes on, the next 8 rows 256). Then the row factors: -e^b |k|^-1, beta e^{b_n - b} |k|^-1,
// scale e^b |q|^-1 (64 floats each) and e^{b_n}.
struct Rec {
    static constexpr int MATRIX = 5120, T = 0, W = 2 * MATRIX, ROWS = 4 * MATRIX, BYTES = ROWS + (3 * C + 4) * 4, STAGE = 21376;
    __device__ static constexpr int panel(int k) { return k * 2048 - k * (k - 1) * 256; }
};
static_assert(10 * BLK * 4 <= 2 * C * 128 && Rec::BYTES % 16 == 0 && Rec::BYTES <= Rec::STAGE && Rec::STAGE % 128 == 0, "");

struct Args {
    GdnParams p;
    const int32_t *cu;
    int rows, num_seqs, V;
    int chunks;                                        // as many as there can be: rows / 64 + num_seqs
    int32_t *first;                                    // [num_seqs + 1] each sequence's first chunk, and their number
    int2 *where;                                       // [chunks] a chunk's first row, and its rows
    unsigned char *records;                            // [chunks][Hv]
    // Long sequences in parts, where there are few:
    int parts;                                         // 1: none
    float *states;                                     // [num_seqs][Hv][2 parts - 1][K][V] what the parts' chains end with
    float *units;                                      // [num_seqs][Hv][2 parts - 1][V] of the states that parts start from, a power of two per column
    float *partial;                                    // [rows (parts - 1) / parts][Hv][V + K] of parts 1 .., outputs and rows of transitions
};

// A sequence of `chunks` chunks in parts: the chunks of each but the last, or 0: it is too short.
constexpr int CUT_CHUNKS = 64, MOST_PARTS = 8;
__device__ __forceinline__ int part_chunks(const Args &a, int chunks) { return a.parts > 1 && chunks >= CUT_CHUNKS ? (chunks + a.parts - 1) / a.parts : 0; }

constexpr int HALF = 2 * C * 128;                      // in shared memory, 64 channels of the chunk's keys, then of its queries

// Matrix descriptors with the 128-byte swizzle, groups of 8 rows at 1024 bytes: the low words (the high one is the same for all).
// K-major: a row of the operand is 128 bytes.
__device__ __forceinline__ uint32_t desc_k(uint32_t at) { return (1u << 16) | (at >> 4); }
// The same bytes with the 128-byte rows along the inner axis (K^T from the tile of K): 64 columns, the next 64 at HALF.
__device__ __forceinline__ uint32_t desc_mn(uint32_t at) { return (static_cast<uint32_t>(HALF >> 4) << 16) | (at >> 4); }
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
// A panel of a record: no swizzle.
__device__ __forceinline__ uint32_t desc_panel(uint32_t at) { return ((128u >> 4) << 16) | (at >> 4); }
constexpr uint32_t PANEL_HIGH = (256u >> 4) | (1u << 14);
// bf16 operands, fp32 sums, 128 rows; `mn`: the second operand is stored along its columns
constexpr uint32_t idesc(int n, bool mn = false)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// d (+)= a b^T, 16 of the inner axis; a in tensor memory
template <uint32_t HIGH = DESC_HIGH>
__device__ __forceinline__ void mma_t(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n"
                 :: "r"(d), "r"(a), "r"(b), "n"(HIGH), "r"(id), "r"(add ? 1u : 0u));
}
// The same with both operands from the same place in shared memory.
__device__ __forceinline__ void mma_gram(uint32_t d, uint32_t ab, uint32_t id, bool add)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%1, %2};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], db, db, %3, p;\n}\n"
                 :: "r"(d), "r"(ab), "n"(DESC_HIGH), "r"(id), "r"(add ? 1u : 0u));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
// The bounds of a sequence; a pair that is no range of the rows has none. *bad: error bits.
__device__ __forceinline__ int2 range(const Args &a, int seq, uint32_t *bad)
{
    const int row = a.cu[seq], end = a.cu[seq + 1];
    if (row >= 0 && end >= row && end <= a.rows) return make_int2(row, end - row);
    *bad |= kErrLengths;
    return make_int2(row, 0);
}

// The chunks of this CTA's chains, one after the other, the same for every warp. A chain: a sequence (longest first), a value head
// and a slice of its columns.
template <bool PARTS>
struct Walk {
    const Args &a;
    const uint16_t *order;
    int item, total, slices;
    int row, left, h, slice;    // of the current chunk: its first row, the chain's rows from there on
    int seq, chunk;
    int kind;                   // 0: from the sequence's state; then for each further part its chain from zeros, and its transition's from the identity
    bool cut = false;           // the sequence is in parts
    int64_t partial = 0;        // the chunk's first row in Args::partial

    __device__ __forceinline__ Walk(const Args &args, const uint16_t *sorted, int vs)
        : a(args), order(sorted), item(blockIdx.x), slices(args.V / vs) { total = args.num_seqs * args.p.Hv * slices * (PARTS ? 2 * args.parts - 1 : 1); }
    // CTA i's chains are i, 2 G - 1 - i, 2 G + i, ..: the longest with the shortest
    __device__ __forceinline__ void advance()
    {
        const int g = gridDim.x, at = item % g;
        item += 2 * (g - 1 - at) + 1;
    }
    // The chain at `item`: whether it has rows (and a slot). *bad: error bits; *all: its rows whatever its slot.
    __device__ __forceinline__ bool chain(uint32_t *bad = nullptr, int *all = nullptr)
    {
        const int kinds = PARTS ? 2 * a.parts - 1 : 1, per = a.p.Hv * slices * kinds, s = item / per, in = (item - s * per) / kinds;
        kind = PARTS ? item % kinds : 0;
        h = in / slices;
        slice = in - h * slices;
        seq = a.num_seqs <= ORDER ? order[s] : s;
        uint32_t e = 0;
        const int2 x = range(a, seq, &e);
        row = x.x;
        left = x.y;
        chunk = a.first[seq];
        if (left > 0 && (left - 1) / C >= a.chunks - chunk) { left = 0; e |= kErrLengths; }   // ranges that overlap: more chunks than rows make
        if (all) *all = kind == 0 ? left : 0;
        if (load_slot(a.p, seq) >= a.p.num_slots) { left = 0; e |= kErrSlotRange; }
        if (bad) *bad = e;
        if (!PARTS) return left > 0;
        const int each = part_chunks(a, (left + C - 1) / C);
        cut = each > 0;
        if (cut) {
            const int64_t ahead = static_cast<int64_t>((kind + 1) / 2) * each * C;
            partial = static_cast<int64_t>(row) * (a.parts - 1) / a.parts + ahead - each * C;
            row += static_cast<int>(ahead < left ? ahead : 0);
            chunk += (kind + 1) / 2 * each;
            left = ahead < left ? (left - static_cast<int>(ahead) < each * C ? left - static_cast<int>(ahead) : each * C) : 0;
        } else if (kind > 0) {
            left = 0;
        }
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
        chunk++;
        if (PARTS) partial += C;
        if (left > 0) return true;
        advance();
        return begin();
    }
    __device__ __forceinline__ int n() const { return left < C ? left : C; }
};

// The rest of a wait whose first try has not come through (out of line: there are many waits, and the instruction cache is small).
// Some twenty warps of a CTA wait at any time and must not take the others' issue slots: the tries sleep (with tests in their place
// 720 us for 640 at 31,516 tokens x 32 heads).
__device__ __noinline__ bool wait_on(uint32_t mbar, uint32_t parity, volatile uint32_t *gave_up, uint32_t *err)
{
    const long long start = clock64();
    while (!phase_over(mbar, parity)) {
        if (*gave_up) return false;
        if (clock64() - start > 4000000000ll) {
            *gave_up = 1;
            if (err) atomicOr(err, kErrTimeout);
            return false;
        }
    }
    return true;
}
// A bounded wait that the CTA gives up as a whole: one that has run out (~2 s) says so to all the others.
struct Waiter {
    volatile uint32_t *gave_up;
    uint32_t *err;
    __device__ __forceinline__ bool operator()(uint32_t mbar, uint32_t parity) const
    {
        return phase_over(mbar, parity) || wait_on(mbar, parity, gave_up, err);
    }
    // by a converged warp, one answer for all lanes
    __device__ __forceinline__ bool warp(uint32_t mbar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, (*this)(mbar, parity));
    }
};

__device__ __forceinline__ constexpr int block_at(int a, int b) { return (a * (a + 1) / 2 + b) * BLK; }

// Chunks are counted up to here: ranges that overlap can have more than 32 bits hold, a workspace (21 KB each) never.
__device__ __forceinline__ int count(int x, int y)
{
    constexpr int MOST = (1 << 30) - 1;
    return x + y < MOST ? x + y : MOST;
}
// One CTA: every sequence's first chunk (their number is not above rows / 64 + num_seqs where the ranges do not overlap; what would
// pass it is left out) and each chunk's rows. Error bits are the chain's.
__global__ void __launch_bounds__(1024) map_kernel(const __grid_constant__ Args a)
{
    __shared__ int sums[32], firsts[1024], starts[1024], lens[1024];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait_then_release();   // no global read before this
    int base = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += 1024) {
        uint32_t bad = 0;
        const int s = s0 + tid;
        const int2 x = s < a.num_seqs ? range(a, s, &bad) : make_int2(0, 0);
        const int n = (x.y + C - 1) / C;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum = count(sum, y);
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        int before = sums[lane];                          // every warp scans the warps' sums
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before = count(before, y);
        }
        const int all = __shfl_sync(0xffffffffu, before, 31), here = warp > 0 ? __shfl_sync(0xffffffffu, before, warp - 1) : 0;
        const int first = count(count(base, here), sum) - n;
        firsts[tid] = first;
        starts[tid] = x.x;
        lens[tid] = x.y;
        if (s < a.num_seqs) a.first[s] = first;
        __syncthreads();
        // each chunk finds its sequence: the last one that begins at it or before it, which has rows
        for (int i = base + tid; i < base + all && i < a.chunks; i += 1024) {
            int low = 0;
#pragma unroll
            for (int step = 512; step > 0; step >>= 1)
                if (firsts[low + step] <= i) low += step;
            const int at = (i - firsts[low]) * C;
            a.where[i] = make_int2(starts[low] + at, lens[low] - at < C ? lens[low] - at : C);
        }
        base = count(base, all);
        __syncthreads();
    }
    if (tid == 0) a.first[a.num_seqs] = base < a.chunks ? base : a.chunks;
}

// T, W and the row factors of a chunk, for the value heads of a key head. Thread t has row t of K K^T (t < 64) or row
// t - 64 of Q K^T, which one product of 128 x 64 gives. A warp's path through the inverse is bound by
// its latencies: as many CTAs an SM as there is shared memory for at K = 128, and registers at 64 (257 sequences of 1 to 342 tokens x 8 heads:
// the three launches 187 us, with six CTAs 189, with five 192; 191 since the increment has three terms).
template <int NH>
__global__ void __launch_bounds__(128, NH == 1 ? 8 : 6) prep_kernel(const __grid_constant__ CUtensorMap tm_qk, const __grid_constant__ Args a)
{
    constexpr int K = 64 * NH;
    // the tiles of q and k; once their products and norms are there, the blocks of A, then of T, on and below the diagonal
    extern __shared__ __align__(1024) unsigned char sm[];
    float *blocks = reinterpret_cast<float *>(sm);
    __shared__ __align__(16) float cols[5 * C];   // b hi, b lo, beta, and of the keys b lo less the logarithm of norm and beta, and e^{p - b} times both
    __shared__ uint64_t bars[2];
    __shared__ uint32_t tmem_at;
    const uint32_t s0 = tc::smem_addr(sm), full = tc::smem_addr(&bars[0]), g_done = tc::smem_addr(&bars[1]);
    const int t = threadIdx.x, lane = t & 31, pw = t >> 5, r = t & 63;
    const bool query = t >= 64;
    const GdnParams &p = a.p;
    const int chunk = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk, per = p.Hv / p.Hk;
    if (t == 0) {
        tc::mbar_init(full, 1);
        tc::mbar_init(g_done, 1);
        tc::prefetch_tensormap(&tm_qk);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no global read before this
    if (chunk >= a.first[a.num_seqs]) return;
    const int2 at = a.where[chunk];
    const int n = at.y;
    if (pw == 0) tc::tmem_alloc<64>(tc::smem_addr(&tmem_at));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = tmem_at;
    if (t == 0) {
        tc::mbar_expect_tx(full, NH * HALF);
#pragma unroll
        for (int hf = 0; hf < NH; hf++) {
            tc::tma_load_2d(s0 + hf * HALF, &tm_qk, (p.Hk + hk) * K + 64 * hf, at.x, full);
            tc::tma_load_2d(s0 + hf * HALF + C * 128, &tm_qk, hk * K + 64 * hf, at.x, full);
        }
    }
    // raw_g (warp 0) and raw_beta (warp 1) of rows 2 lane, 2 lane + 1
    float in0 = 0.f, in1 = 0.f, rate = 0.f, dtb = 0.f;
    auto fetch = [&](int h) {
        if (pw < 2) {
            const uint16_t *from = pw == 0 ? p.rg : p.rb;
            const int64_t ld = pw == 0 ? p.ld_g : p.ld_beta, row = static_cast<int64_t>(at.x) + 2 * lane;
            if (2 * lane < n) in0 = bf16_to_f32(from[row * ld + h]);
            if (2 * lane + 1 < n) in1 = bf16_to_f32(from[(row + 1) * ld + h]);
            if (pw == 0) {
                rate = p.A_log[h];
                dtb = p.dt_bias ? p.dt_bias[h] : 0.f;
            }
        }
    };
    fetch(hk * per);
    bool ok = tc::mbar_wait(full, 0);
    if (pw == 0) {
        if (elect_one()) {
#pragma unroll
            for (int k = 0; k < K / 16; k++) mma_gram(tmem, desc_k(s0 + (k / 4) * HALF + (k % 4) * 32), idesc(C), k > 0);
            tc::commit(g_done);
        }
        __syncwarp();
    }
    // the norm of this thread's row
    float norm = 0.f;
    if (r < n) {
        float2 sum = make_float2(0.f, 0.f);
        const unsigned char *own = sm + t * 128;
#pragma unroll
        for (int hf = 0; hf < NH; hf++)
#pragma unroll
            for (int x = 0; x < 8; x++) {
                const uint4 q = *reinterpret_cast<const uint4 *>(own + hf * HALF + ((x ^ (t & 7)) << 4));
                const uint32_t qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    const float2 f = make_float2(__uint_as_float(qq[y] << 16), __uint_as_float(qq[y] & 0xffff0000u));
                    sum = ffma2(f, f, sum);
                }
            }
        norm = rsqrtf(sum.x + sum.y + p.eps);
    }
    ok &= tc::mbar_wait(g_done, 0);
    tc::fence_after_sync();
    for (int h = hk * per; h < (hk + 1) * per; h++) {
        unsigned char *rec = a.records + (static_cast<int64_t>(chunk) * p.Hv + h) * Rec::BYTES;
        float *set = reinterpret_cast<float *>(rec + Rec::ROWS);
        if (pw == 0) {                                                    // the running decay, in units of log 2
            rate = expf(rate) * -1.44269504f;
            const float g0 = 2 * lane < n ? bounded(rate * softplus_f(in0 + dtb)) : 0.f, g1 = 2 * lane + 1 < n ? bounded(rate * softplus_f(in1 + dtb)) : 0.f;
            const FixedDecay f0 = FixedDecay::of(g0), f1 = FixedDecay::of(g1), b = (f0 + f1).up_to(32);
            const bool nan = any_below(g0 != g0 || g1 != g1) || g0 != g0;
            const float2 x0 = FixedDecay{b.hi - f1.hi, b.lo - f1.lo}.get(nan), x1 = b.get(nan || g1 != g1);
            *reinterpret_cast<float2 *>(cols + 2 * lane) = make_float2(x0.x, x1.x);
            *reinterpret_cast<float2 *>(cols + C + 2 * lane) = make_float2(x0.y, x1.y);
        } else if (pw == 1) {
            *reinterpret_cast<float2 *>(cols + 2 * C + 2 * lane) =
                make_float2(2 * lane < n ? sigmoid_f(in0) : 0.f, 2 * lane + 1 < n ? sigmoid_f(in1) : 0.f);
        }
        if (h + 1 < (hk + 1) * per) fetch(h + 1);
        __syncthreads();
        const float b_hi = cols[r], b_lo = cols[C + r];
        const float scale = (query ? p.scale : 1.f) * norm;
        if (!query) {
            const float e_hi = cols[C - 1], e_lo = cols[2 * C - 1], own = norm * cols[2 * C + r];
            set[r] = -ex2(b_hi + b_lo) * norm;
            set[C + r] = ex2((e_hi - b_hi) + (e_lo - b_lo)) * own;
            if (r == 0) set[3 * C] = ex2(e_hi + e_lo);
            cols[3 * C + r] = b_lo - (r < n ? __log2f(own) : 0.f);
            cols[4 * C + r] = ex2((cols[r | 15] - b_hi) + (cols[C + (r | 15)] - b_lo)) * own;
        } else {
            set[2 * C + r] = p.scale * ex2(b_hi + b_lo) * norm;
        }
        __syncthreads();
        // row r of A (its blocks up to the diagonal's), or of W
        const int low = (pw & 1) * 2;                                         // the first block with a diagonal in the warp's rows
        const uint32_t tg = tmem + (static_cast<uint32_t>(pw * 32) << 16);
        float2 d[8];
        auto put = [&](int bl) {
            if (bl > r >> 4) return;
            if (query) {
                unsigned char *to = rec + Rec::W + Rec::panel(bl) + ((r - 16 * bl) >> 3) * 256 + (r & 7) * 16;
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) split2(d[4 * y + i].x, d[4 * y + i].y, hi[i], lo[i]);
                    *reinterpret_cast<uint4 *>(to + y * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(to + Rec::MATRIX + y * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            } else {
                float *to = blocks + block_at(r >> 4, bl) + (r & 15) * 20;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    *reinterpret_cast<float4 *>(to + 4 * i) = make_float4(d[2 * i].x, d[2 * i].y, d[2 * i + 1].x, d[2 * i + 1].y);
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
            if (r >= n) {                                                     // not a row of the chunk: whatever it held
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
        __syncthreads();
        const int gq = lane >> 2, tq = lane & 3;
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
        __syncthreads();
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
            __syncthreads();                                                       // A has been read
#pragma unroll
            for (int x = 0; x < 4; x++) {
                const int col = gq + 8 * (x >> 1), row = 8 * hf + 2 * tq + (x & 1);
                A[row * 20 + col] = out[x];
            }
        }
        __syncthreads();
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
            __syncthreads();                                                       // A has been read
            float *at = blocks + block_at(2 + hf, mt);
#pragma unroll
            for (int rt = 0; rt < 2; rt++)
#pragma unroll
                for (int x = 0; x < 4; x++) at[(8 * rt + 2 * tq + (x & 1)) * 20 + gq + 8 * (x >> 1)] = out[rt][x];
        }
        __syncthreads();
        // T - I, hi and lo: half of row r
#pragma unroll 1
        for (int bl = t >> 6 << 1; bl <= r >> 4 && bl < (t >> 6 << 1) + 2; bl++) {
            const float *from = blocks + block_at(r >> 4, bl) + (r & 15) * 20;
            unsigned char *to = rec + Rec::T + Rec::panel(bl) + ((r - 16 * bl) >> 3) * 256 + (r & 7) * 16;
#pragma unroll
            for (int y = 0; y < 2; y++) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float4 x = *reinterpret_cast<const float4 *>(from + 8 * y + 4 * i);
                    const int one = r - bl * 16 - 8 * y - 4 * i;                  // the diagonal's column of the four
                    x.x = one == 0 ? 0.f : x.x; x.y = one == 1 ? 0.f : x.y; x.z = one == 2 ? 0.f : x.z; x.w = one == 3 ? 0.f : x.w;
                    split2(x.x, x.y, hi[2 * i], lo[2 * i]);
                    split2(x.z, x.w, hi[2 * i + 1], lo[2 * i + 1]);
                }
                *reinterpret_cast<uint4 *>(to + y * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + Rec::MATRIX + y * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        __syncthreads();                                                      // blocks and columns are free again
    }
    if (!ok) {                                             // no CTA ends with copies or MMAs in flight
        if (p.err) atomicOr(p.err, kErrTimeout);
        (void)tc::mbar_wait(full, 0);
        (void)tc::mbar_wait(g_done, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (pw == 0) tc::tmem_dealloc<64>(tmem);
}
// ---- the chains ---------------------------------------------------------------------------

// warps 0 - 15 the chain, 16 - 19 outputs, 20 copies, 22 the rows behind a sequence's end, 23 MMAs. A warp reads the quarter of tensor
// memory that its number modulo 4 names and runs on that quarter of the multiprocessor: with halves of the value columns the chain's are 0
// and 1, and the MMAs' warp stays out of their way (16,384 tokens x 32 heads in one part 764 us, as warp 21 781).
constexpr int THREADS = 768;
constexpr int STAGES = 3;          // chunks in shared memory
struct Smem {
    static constexpr int QK = 2 * HALF, V = C * 256;
    static constexpr int REC = QK + V, STAGE = QK + V + Rec::STAGE;
    static constexpr int SORT = STAGES * STAGE, BARS = SORT + ORDER * 2, NBARS = 3 * STAGES + 14, END = BARS + NBARS * 8 + 16;
};
static_assert(Smem::STAGE % 128 == 0 && Smem::END <= 232448, "shared memory of a CTA");

// columns of tensor memory
constexpr uint32_t T_S = 0;      // first operand of K S and Q S: the quarters of the channels one after the other, each hi | lo; then the state's increment
constexpr uint32_t T_Y = 128;    // K S; then Y, later Z scaled, as operands, by quarters of the rows, each hi | lo
constexpr uint32_t T_Z = 192;    // Y, to which its product is added: Z; then as an operand, the same way
constexpr uint32_t T_O = 256;    // Q S and W Z
constexpr uint32_t T_3 = 384;    // the scaled Z's third terms

// Value columns VS at a time (a slice of V), a thread with one of them and a quarter of the channels, or of the rows. PARTS: long sequences are in parts.
template <int NH, int VS, bool PARTS>
__global__ void __launch_bounds__(THREADS, 1)
chain_kernel(const __grid_constant__ CUtensorMap tm_qk, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args a)
{
    constexpr int K = 64 * NH, KP = K / 4, VW = VS / 32;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = tc::smem_addr(sm), b0 = s0 + Smem::BARS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto full = [&](int s) { return b0 + s * 8; };                          // a chunk has landed
    auto empty = [&](int s) { return b0 + (STAGES + s) * 8; };              // and is no longer needed
    auto clean = [&](int s) { return b0 + (2 * STAGES + s) * 8; };          // its keys behind the sequence's end are zeros
    const uint32_t bx = b0 + 3 * STAGES * 8;
    const uint32_t s_hi = bx, s_lo = bx + 8, ks_done = bx + 16, y_hi = bx + 24, y_lo = bx + 32, z_done = bx + 40, z_hi = bx + 48, z_lo = bx + 56,
                   w_ready = bx + 64, s_done = bx + 72, o_done = bx + 80, o_free = bx + 88, drained = bx + 96, z_3 = bx + 104;
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(sm + Smem::BARS + Smem::NBARS * 8);   // tensor memory's base, whether a wait has given up
    uint16_t *order = reinterpret_cast<uint16_t *>(sm + Smem::SORT);
    const GdnParams &p = a.p;

    if (tid == 0) {
        for (int i = 0; i < STAGES; i++) {
            tc::mbar_init(full(i), 1);
            tc::mbar_init(empty(i), 2 + VW);                           // the MMAs, the outputs' warps and the one that clears keys
            tc::mbar_init(clean(i), 1);
        }
        for (const uint32_t b : {s_hi, s_lo, y_hi, y_lo, z_hi, z_lo, z_3, w_ready}) tc::mbar_init(b, 4 * VW);
        tc::mbar_init(ks_done, 1);
        tc::mbar_init(z_done, 1);
        tc::mbar_init(s_done, 1);
        tc::mbar_init(o_done, 1);
        tc::mbar_init(o_free, VW);
        tc::mbar_init(drained, 1);
        words[1] = 0;
        tc::prefetch_tensormap(&tm_qk);
        tc::prefetch_tensormap(&tm_v);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no global read before this
    // the sequences by falling length: each finds its place
    if (a.num_seqs <= ORDER) {
        int *len = reinterpret_cast<int *>(sm);           // the first stage's place
        for (int i = tid; i < a.num_seqs; i += THREADS) {
            uint32_t bad = 0;
            len[i] = range(a, i, &bad).y;
        }
        __syncthreads();
        for (int i = tid; i < a.num_seqs; i += THREADS) {
            const int own = len[i];
            int before = 0;
            for (int k = 0; k < a.num_seqs; k++) before += len[k] > own || (len[k] == own && k < i);
            order[before] = static_cast<uint16_t>(i);
        }
        tc::fence_proxy_async();                          // the place is TMA's from here on
    }
    if (warp == 23) tc::tmem_alloc<512>(s0 + Smem::BARS + Smem::NBARS * 8);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = words[0];
    const Waiter wait{words + 1, p.err};
    Walk<PARTS> w(a, order, VS);

    if (warp < 16) {
        // ---- the chain ----
        const int quarter = warp & 3, part = warp >> 2;                       // of the value columns; of the channels and rows
        if (quarter < VW) {
            const int j = quarter * 32 + lane;                                // this thread's value column in the slice
            const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t ts = t0 + T_S + part * KP, ty = t0 + T_Y + part * 16, tz = t0 + T_Z + part * 16, t3 = t0 + T_3 + part * 8;
            float2 S[KP / 2];                                                 // channels KP part .. of column j
            auto give = [&](uint32_t mbar) {                                  // what the products wait for is in tensor memory
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(mbar);
            };
            // Operands are given term by term: the products of the first are under way while the second is formed.
            auto give_s = [&] {
                uint32_t hi[KP / 2];
#pragma unroll
                for (int i = 0; i < KP / 2; i++) hi[i] = pack_bf16x2(S[i].x, S[i].y);
#pragma unroll
                for (int i = 0; i < KP / 2; i += 8) tmem_st8(ts + i, *reinterpret_cast<const uint32_t(*)[8]>(hi + i));
                give(s_hi);
#pragma unroll
                for (int i = 0; i < KP / 2; i += 8) {
                    uint32_t lo[8];
#pragma unroll
                    for (int x = 0; x < 8; x++) lo[x] = rest2(S[i + x].x, S[i + x].y, hi[i + x]);
                    tmem_st8(ts + KP / 2 + i, lo);
                }
                give(s_lo);
            };
            bool more = w.begin(), first = true;
            for (uint32_t c = 0; more; c++) {
                const int s = c % STAGES, n = w.n();
                const uint32_t one = c & 1;
                const unsigned char *stage = sm + s * Smem::STAGE;
                float *tile = nullptr;
                bool write = false;
                const bool last = w.left <= C, transition = PARTS && w.kind > 0 && w.kind % 2 == 0;
                if (first || last) {
                    const int64_t slot = load_slot(p, w.seq);
                    if (slot >= 0) tile = p.pool + slot * p.slot_stride + (static_cast<int64_t>(w.h) * K + part * KP) * a.V + w.slice * VS + j;
                    write = slot >= 0 && slot != p.null_slot;
                }
                if (first) {
                    if (PARTS && w.kind > 0) tile = nullptr;
#pragma unroll
                    for (int i = 0; i < KP / 2; i++) {
                        S[i] = tile ? make_float2(tile[static_cast<int64_t>(2 * i) * a.V], tile[static_cast<int64_t>(2 * i + 1) * a.V]) : make_float2(0.f, 0.f);
                        if (transition) S[i] = make_float2(part * KP + 2 * i == j ? 1.f : 0.f, part * KP + 2 * i + 1 == j ? 1.f : 0.f);
                    }
                    give_s();
                }
                if (PARTS && last && w.cut) {   // the parts are joined later
                    tile = a.states + ((static_cast<int64_t>(w.seq) * p.Hv + w.h) * (2 * a.parts - 1) + w.kind) * K * a.V + part * KP * a.V + j;
                    write = true;
                }
                // v of this column and quarter of the rows
                if (!wait.warp(full(s), (c / STAGES) & 1)) break;
                uint32_t v[8];
                {
                    const unsigned char *at = stage + Smem::QK + part * 16 * (VS * 2) + j * 2;
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        v[i] = transition ? 0u : *reinterpret_cast<const uint16_t *>(at + 2 * i * VS * 2) |
                               static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(at + (2 * i + 1) * VS * 2)) << 16;
                }
                const float *set = reinterpret_cast<const float *>(stage + Smem::REC + Rec::ROWS);
                const float gamma = set[3 * C];
                // Y = V - e^b K^ S; rows past the chunk's end are zeros, whatever is in memory there
                if (!wait.warp(ks_done, one)) break;
                tc::fence_after_sync();
                {
                    uint32_t x[16];
                    float2 y[8];
                    tmem_ld(ty, x);
                    const float4 *ys = reinterpret_cast<const float4 *>(set + part * 16);
                    tc::tmem_ld_wait();
                    if (n - part * 16 < 16) {
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            if (part * 16 + e >= n) {
                                x[e] = 0u;
                                v[e / 2] &= e % 2 ? 0x0000ffffu : 0xffff0000u;
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const float4 f = ys[e / 2];
                        y[e] = ffma2(e % 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y), make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                     make_float2(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u)));
                    }
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) hi[e] = pack_bf16x2(y[e].x, y[e].y);
                    tmem_st8(ty, hi);
                    // Z's sums begin with Y (the products that read the last chunk's operand there are over when K S is)
#pragma unroll
                    for (int e = 0; e < 8; e += 4)
                        tmem_st8(tz + 2 * e, {__float_as_uint(y[e].x), __float_as_uint(y[e].y), __float_as_uint(y[e + 1].x), __float_as_uint(y[e + 1].y),
                                              __float_as_uint(y[e + 2].x), __float_as_uint(y[e + 2].y), __float_as_uint(y[e + 3].x), __float_as_uint(y[e + 3].y)});
                    give(y_hi);
#pragma unroll
                    for (int e = 0; e < 8; e++) lo[e] = rest2(y[e].x, y[e].y, hi[e]);
                    tmem_st8(ty + 8, lo);
                    give(y_lo);
                }
                // Z scaled, for the state, in three terms (with two the states were off by 2.5e-6 of their norm instead of 1.1e-6 to 1.4e-6, 31,516 tokens x 32 heads
                // 544 us instead of 569; with two, and T's diagonal in the products, 4.5e-6 and 550), and then as it is, for the outputs
                if (!wait.warp(z_done, one)) break;
                tc::fence_after_sync();
                {
                    uint32_t x[16], hi[8], lo[8];
                    float2 z[8];
                    tmem_ld(tz, x);
                    const float4 *zs = reinterpret_cast<const float4 *>(set + C + part * 16);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const float4 f = zs[e / 2];
                        z[e] = fmul2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), e % 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
                        hi[e] = pack_bf16x2(z[e].x, z[e].y);
                    }
                    tmem_st8(ty, hi);
                    give(z_hi);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        z[e] = left(z[e], hi[e]);
                        lo[e] = pack_bf16x2(z[e].x, z[e].y);
                    }
                    tmem_st8(ty + 8, lo);
                    if (NH == 2) give(z_lo);               // at K = 64 the products take no longer than a barrier: the second term with the third
#pragma unroll
                    for (int e = 0; e < 8; e++) lo[e] = rest2(z[e].x, z[e].y, lo[e]);
                    tmem_st8(t3, lo);
                    give(z_3);
                    tmem_ld(tz, x);                        // again: it is not kept in registers meanwhile
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; e++) split2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), hi[e], lo[e]);
                    tmem_st8(tz, hi);
                    tmem_st8(tz + 8, lo);
                    give(w_ready);
                }
                // S <- gamma S + its increment
                more = w.next();
                if (!wait.warp(s_done, one)) break;
                tc::fence_after_sync();
                const float2 g2 = make_float2(gamma, gamma);
#pragma unroll
                for (int i = 0; i < KP / 2; i += 8) {
                    uint32_t x[16];
                    tmem_ld(ts + 2 * i, x);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; e++) S[i + e] = ffma2(g2, S[i + e], make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])));
                }
                first = last;
                if (!last) {
                    give_s();
                } else if (write) {
#pragma unroll
                    for (int i = 0; i < KP / 2; i++) {
                        tile[static_cast<int64_t>(2 * i) * a.V] = S[i].x;
                        tile[static_cast<int64_t>(2 * i + 1) * a.V] = S[i].y;
                    }
                }
            }
        }
    } else if (warp < 20) {
        // ---- outputs ----
        const int quarter = warp & 3, j = quarter * 32 + lane;
        // chains that are skipped: their error bits, and zeros for a slot past the pool
        for (Walk<PARTS> z(a, order, VS); z.item < z.total; z.advance()) {
            uint32_t bad;
            int all;
            z.chain(&bad, &all);
            if (!bad) continue;
            if (p.err && quarter == 0 && lane == 0) atomicOr(p.err, bad);
            if (j < VS)
                for (int i = 0; i < all; i++)
                    p.out[(static_cast<int64_t>(z.row) + i) * p.ld_out + static_cast<int64_t>(z.h) * a.V + z.slice * VS + j] = 0;
        }
        if (quarter < VW) {
            const uint32_t t0 = tmem + T_O + (static_cast<uint32_t>(quarter * 32) << 16);
            bool more = w.begin();
            for (uint32_t c = 0; more; c++) {
                const int s = c % STAGES, n = w.n();
                uint16_t *out = p.out + static_cast<int64_t>(w.row) * p.ld_out + static_cast<int64_t>(w.h) * a.V + w.slice * VS + j;
                const float *qs = reinterpret_cast<const float *>(sm + s * Smem::STAGE + Smem::REC + Rec::ROWS) + 2 * C;
                float *part = PARTS && w.kind > 0 ? a.partial + (w.partial * p.Hv + w.h) * (a.V + K) + (w.kind % 2 ? 0 : a.V) + j : nullptr;
                more = w.next();
                if (!wait.warp(o_done, c & 1)) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int i = 0; i < C; i += 16) {
                    uint32_t x[16], y[16];
                    tmem_ld(t0 + i, x);
                    tmem_ld(t0 + C + i, y);
                    tc::tmem_ld_wait();
                    if (i == C - 16) {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive(o_free);
                    }
                    auto store = [&](auto whole) {
#pragma unroll
                        for (int r = 0; r < 16; r += 2) {
                            const float2 o = ffma2(*reinterpret_cast<const float2 *>(qs + i + r), make_float2(__uint_as_float(x[r]), __uint_as_float(x[r + 1])),
                                                   make_float2(__uint_as_float(y[r]), __uint_as_float(y[r + 1])));
                            const uint32_t o2 = pack_bf16x2(o.x, o.y);
                            if (whole || i + r < n) *out = static_cast<uint16_t>(o2);
                            out += p.ld_out;
                            if (whole || i + r + 1 < n) *out = static_cast<uint16_t>(o2 >> 16);
                            out += p.ld_out;
                        }
                    };
                    if (PARTS && part) {
                        const int64_t ld = static_cast<int64_t>(p.Hv) * (a.V + K);
                        auto keep = [&](auto whole) {
#pragma unroll
                            for (int r = 0; r < 16; r += 2) {
                                const float2 o = ffma2(*reinterpret_cast<const float2 *>(qs + i + r), make_float2(__uint_as_float(x[r]), __uint_as_float(x[r + 1])),
                                                       make_float2(__uint_as_float(y[r]), __uint_as_float(y[r + 1])));
                                if (whole || i + r < n) *part = o.x;
                                part += ld;
                                if (whole || i + r + 1 < n) *part = o.y;
                                part += ld;
                            }
                        };
                        if (i + 16 <= n) keep(std::true_type{});
                        else keep(std::false_type{});
                    } else if (i + 16 <= n) store(std::true_type{});
                    else store(std::false_type{});
                }
                __syncwarp();
                if (lane == 0) arrive(empty(s));
            }
        }
    } else if (warp == 20) {
        // ---- copies ----
        if (lane == 0) {
            const int per = p.Hv / p.Hk;
            bool more = w.begin();
            uint32_t c = 0;
            for (; more; c++) {
                const int s = c % STAGES;
                if (c >= STAGES && !wait(empty(s), (c / STAGES - 1) & 1)) break;
                const uint32_t at = s0 + s * Smem::STAGE;
                tc::mbar_expect_tx(full(s), NH * HALF + C * VS * 2 + Rec::BYTES);
#pragma unroll
                for (int hf = 0; hf < NH; hf++) {
                    const int x = w.h / per * K + 64 * hf;
                    tc::tma_load_2d(at + hf * HALF, &tm_qk, p.Hk * K + x, w.row, full(s));
                    tc::tma_load_2d(at + hf * HALF + C * 128, &tm_qk, x, w.row, full(s));
                }
                tc::tma_load_2d(at + Smem::QK, &tm_v, 2 * p.Hk * K + w.h * a.V + w.slice * VS, w.row, full(s));
                tc::bulk_g2s(at + Smem::REC, a.records + (static_cast<int64_t>(w.chunk) * p.Hv + w.h) * Rec::BYTES, Rec::BYTES, full(s));
                more = w.next();
            }
            // no CTA ends with copies in flight
            for (uint32_t k = c > STAGES ? c - STAGES : 0; k < c; k++) (void)tc::mbar_wait(full(k % STAGES), (k / STAGES) & 1);
        }
    } else if (warp == 23) {
        // ---- MMAs ----
        bool more = w.begin();
        for (uint32_t c = 0; more; c++) {
            const int s = c % STAGES;
            const uint32_t one = c & 1, at = s0 + s * Smem::STAGE, rec = at + Smem::REC;
            if (!wait.warp(full(s), (c / STAGES) & 1) || !wait.warp(s_hi, one)) break;
            tc::fence_after_sync();
            // a term (x) of S^T times the keys or the queries (the rows `from` on)
            auto times_s = [&](uint32_t d, uint32_t from, int x) {
#pragma unroll
                for (int k = 0; k < K / 16; k++)
                    mma_t(d, tmem + T_S + k / (KP / 16) * KP + x * (KP / 2) + k % (KP / 16) * 8, desc_k(from + (k / 4) * HALF + (k % 4) * 32), idesc(C), x + k > 0);
            };
            // a term of a record's matrix (y) times one (x) of Y or Z; rows before 16 k are zero in columns 16 k ..
            auto times_rec = [&](uint32_t d, uint32_t from, uint32_t matrix, int x, int y, bool first) {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma_t<PANEL_HIGH>(d + 16 * k, from + k * 16 + x * 8, desc_panel(matrix + y * Rec::MATRIX + Rec::panel(k)), idesc(C - 16 * k), !first || k > 0);
            };
            if (elect_one()) times_s(tmem + T_Y, at, 0);
            __syncwarp();
            if (!wait.warp(s_lo, one)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                times_s(tmem + T_Y, at, 1);
                tc::commit(ks_done);
            }
            __syncwarp();
            if (c > 0 && !wait.warp(o_free, one ^ 1)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                times_s(tmem + T_O, at + C * 128, 0);
                times_s(tmem + T_O, at + C * 128, 1);
            }
            __syncwarp();
            if (!wait.warp(y_hi, one)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                times_rec(tmem + T_Z, tmem + T_Y, rec + Rec::T, 0, 0, false);
                times_rec(tmem + T_Z, tmem + T_Y, rec + Rec::T, 0, 1, false);
            }
            __syncwarp();
            if (!wait.warp(y_lo, one)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                times_rec(tmem + T_Z, tmem + T_Y, rec + Rec::T, 1, 0, false);
                tc::commit(z_done);
            }
            __syncwarp();
            // the state's increment
            auto increment = [&](int x) {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma_t(tmem + T_S, x < 2 ? tmem + T_Y + k * 16 + x * 8 : tmem + T_3 + k * 8, desc_mn(at + k * 16 * 128), idesc(K, true), x + k > 0);
            };
            if (!wait.warp(z_hi, one) || (w.left < C && !wait.warp(clean(s), (c / STAGES) & 1))) break;
            tc::fence_after_sync();
            if (elect_one()) increment(0);
            __syncwarp();
            if (!wait.warp(NH == 2 ? z_lo : z_3, one)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                increment(1);
            }
            __syncwarp();
            if (NH == 2 && !wait.warp(z_3, one)) break;
            if (NH == 2) tc::fence_after_sync();
            if (elect_one()) {
                increment(2);
                tc::commit(s_done);
            }
            __syncwarp();
            if (!wait.warp(w_ready, one)) break;
            tc::fence_after_sync();
            if (elect_one()) {
                times_rec(tmem + T_O + C, tmem + T_Z, rec + Rec::W, 0, 0, true);
                times_rec(tmem + T_O + C, tmem + T_Z, rec + Rec::W, 1, 0, false);
                times_rec(tmem + T_O + C, tmem + T_Z, rec + Rec::W, 0, 1, false);
                tc::commit(empty(s));
                tc::commit(o_done);
            }
            __syncwarp();
            more = w.next();
        }
        // nor with MMAs
        if (elect_one()) tc::commit(drained);
        __syncwarp();
        (void)tc::mbar_wait(drained, 0);
    } else if (warp == 22) {
        // ---- keys behind a sequence's end: another sequence's, and 0 times what they may hold is not 0; the next chain's state to L2 ----
        bool more = w.begin();
        Walk<PARTS> z(a, order, VS);
        bool another = z.begin();
        int item = -1;
        for (uint32_t c = 0; more; c++) {
            const int s = c % STAGES, n = w.n();
            if (!wait.warp(full(s), (c / STAGES) & 1)) break;
            if (n < C) {
                for (int i = n * 8 + lane; i < C * 8; i += 32)
#pragma unroll
                    for (int hf = 0; hf < NH; hf++) *reinterpret_cast<uint4 *>(sm + s * Smem::STAGE + hf * HALF + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                tc::fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                arrive(clean(s));
                arrive(empty(s));   // the stage is held until here: this warp cannot fall behind by a turn of the ring
            }
            // the walks past sequences without rows come after what others wait for
            if (w.item != item) {
                item = w.item;
                if (another) { z.advance(); another = z.begin(); }
                const int64_t slot = another && (!PARTS || z.kind == 0) ? load_slot(p, z.seq) : -1;
                if (slot >= 0) {
                    const float *tile = p.pool + slot * p.slot_stride + static_cast<int64_t>(z.h) * K * a.V + z.slice * VS;
                    for (int i = lane; i < K * VW; i += 32)
                        asm volatile("prefetch.global.L2 [%0];" :: "l"(tile + static_cast<int64_t>(i / VW) * a.V + i % VW * 32));
                }
            }
            more = w.next();
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 23) tc::tmem_dealloc<512>(tmem);
}

// ---- joining the parts ----------------------------------------------------------------------
// A part's tokens take the state it starts from, S, to A S + B: B is where its chain from zeros ends, A (its transition) where the one from the
// identity with v = 0 does. An output is that chain's own and the transition's row times S.

// The unit of values up to `top`, a power of two that puts them into fp16's upper range (2^13 and more), within what fp32 and its reciprocal hold.
__device__ __forceinline__ float unit_of(float top)
{
    const int e = static_cast<int>(__float_as_uint(top) >> 23 & 255);
    return __int_as_float(((e < 16 ? 16 : e > 254 ? 254 : e) - 13) << 23);
}
// One over a power of two.
__device__ __forceinline__ float over(float unit) { return __int_as_float(0x7f000000 - __float_as_int(unit)); }
// The larger of `top` and |x|, where that is finite.
__device__ __forceinline__ float with(float top, float x) { return fabsf(x) > top && fabsf(x) <= 3.4028234e38f ? fabsf(x) : top; }
// A CTA per (sequence, value head, 32 value columns): each part's end from its start, in order; the last is the sequence's. A thread has a
// column and K / 8 channels. The next part's transition is on its way while one is applied.
template <int K>
__global__ void __launch_bounds__(256) ends_kernel(const __grid_constant__ Args a)
{
    constexpr int R = K / 8;
    extern __shared__ __align__(1024) unsigned char sm[];
    float *start = reinterpret_cast<float *>(sm), *trans = start + K * 32, *most = trans + 2 * K * K;   // [K][32], [2][K][K], [8][32]
    const GdnParams &p = a.p;
    const int slices = K / 32, slice = blockIdx.x % slices, h = blockIdx.x / slices % p.Hv, seq = blockIdx.x / slices / p.Hv, kinds = 2 * a.parts - 1;
    const int tid = threadIdx.x, v = tid % 32, warp = tid / 32, c0 = warp * R;
    pdl_wait_then_release();   // no global read before this
    uint32_t bad = 0;
    const int2 x = range(a, seq, &bad);
    const int chunks = (x.y + C - 1) / C, each = part_chunks(a, chunks);
    const int64_t slot = load_slot(p, seq), at = static_cast<int64_t>(seq) * p.Hv + h;
    if (each == 0 || slot >= p.num_slots || chunks > a.chunks - a.first[seq]) return;
    float *states = a.states + at * kinds * K * K, *own = states + c0 * K + slice * 32 + v, *units = a.units + at * kinds * K + slice * 32 + v;
    auto fetch = [&](int part) {
        if (part * each < chunks) {
            const float *from = states + 2 * part * K * K;
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(trans + part % 2 * K * K));
#pragma unroll
            for (int i = 0; i < K * K / 1024; i++) cp_async16(to + (tid + 256 * i) * 16, from + (tid + 256 * i) * 4, true);
        }
        cp_async_commit();
    };
    fetch(1);
    float s[R];
#pragma unroll
    for (int c = 0; c < R; c++) s[c] = own[c * K];
    for (int part = 1; part * each < chunks; part++) {
        float *B = own + (2 * part - 1) * K * K;
        float next[R], top = 0.f;
#pragma unroll
        for (int c = 0; c < R; c++) {
            next[c] = B[c * K];
            start[(c0 + c) * 32 + v] = s[c];
            top = with(top, s[c]);
        }
        most[warp * 32 + v] = top;
        cp_async_wait_all();                               // this part's transition
        __syncthreads();
        fetch(part + 1);
        if (warp == 0) {                                   // the columns' largest finite values
            for (int i = 1; i < 8; i++) top = fmaxf(top, most[i * 32 + v]);
            units[(part == 1 ? 0 : 2 * part - 3) * K] = unit_of(top);
        }
        const float *A = trans + part % 2 * K * K + c0 * K;
#pragma unroll 2
        for (int k = 0; k < K; k += 4) {
            const float x0 = start[k * 32 + v], x1 = start[(k + 1) * 32 + v], x2 = start[(k + 2) * 32 + v], x3 = start[(k + 3) * 32 + v];
#pragma unroll
            for (int c = 0; c < R; c++) {
                const float4 f = *reinterpret_cast<const float4 *>(A + c * K + k);
                next[c] = fmaf(f.x, x0, fmaf(f.y, x1, fmaf(f.z, x2, fmaf(f.w, x3, next[c]))));
            }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < R; c++) {
            s[c] = next[c];
            B[c * K] = s[c];
        }
    }
    cp_async_wait_all();
    if (slot >= 0 && slot != p.null_slot) {
        float *to = p.pool + slot * p.slot_stride + static_cast<int64_t>(h) * K * K + c0 * K + slice * 32 + v;
#pragma unroll
        for (int c = 0; c < R; c++) to[c * K] = s[c];
    }
}

// d += a b, 16 rows by 8 columns, 16 of the inner axis
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A CTA per (two chunks, value head): the outputs of chunks of parts 1 .., 16 rows a warp, by fp16 products: 2^-12 of a term, where the
// outputs are rounded to 2^-9. fp16's range is short, and both factors shrink with the decays over a part: a transition's rows are in units of
// their own largest values, the states in those of their columns'. The rows are copied to shared memory whole, so that they are on chip for both their largest
// values and the products (read again from L1 instead 10 us more). The CTAs of the first parts' chunks, which have nothing to do, take turns with the others.
template <int K>
__global__ void __launch_bounds__(256, 2) outputs_kernel(const __grid_constant__ Args a)
{
    constexpr int LD = K + 4;                              // pairs of a row of the state; with its columns' bit 1 turned in half of the rows, no bank conflicts
    constexpr int ROW = K + 16;                            // floats from one row of a transition to the next: no bank conflicts
    extern __shared__ __align__(1024) unsigned char sm[];
    uint32_t *state = reinterpret_cast<uint32_t *>(sm);    // [K / 2][LD]: of two rows each, fp16
    float *rows = reinterpret_cast<float *>(state + K / 2 * LD) + (threadIdx.x >> 5) * 16 * ROW;   // this warp's 16 of the transitions
    __shared__ __align__(16) float units[K];
    const GdnParams &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.x % p.Hv, kinds = 2 * a.parts - 1;
    const int pairs = gridDim.x / p.Hv, pair_at = blockIdx.x / p.Hv, pair = pair_at & 1 ? pair_at >> 1 : (pairs >> 1) + (pair_at >> 1);
    pdl_wait_then_release();   // no global read before this
    // the two chunks' states, where they are joined (NULL: not), and of this warp's the sequence, its row and its place among the partial outputs
    const float *from[2], *unit[2];
    int2 own = make_int2(0, 0);
    int row = 0;
    const float *mine = nullptr;
    const int64_t ld = static_cast<int64_t>(p.Hv) * 2 * K;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int chunk = 2 * pair + i;
        from[i] = unit[i] = nullptr;
        if (chunk >= a.first[a.num_seqs]) continue;
        int seq = 0;
        while (seq + 1 < a.num_seqs && a.first[seq + 1] <= chunk) seq++;
        uint32_t bad = 0;
        const int2 x = range(a, seq, &bad);
        const int chunks = (x.y + C - 1) / C, each = part_chunks(a, chunks), at = chunk - a.first[seq];
        if (each == 0 || at < each || at >= chunks || chunks > a.chunks - a.first[seq] || load_slot(p, seq) >= p.num_slots) continue;
        const int part = at / each;
        const int64_t start = (static_cast<int64_t>(seq) * p.Hv + h) * kinds + (part == 1 ? 0 : 2 * part - 3);
        from[i] = a.states + start * K * K;
        unit[i] = a.units + start * K;
        if (warp / 4 == i) {
            own = x;
            row = at * C + warp % 4 * 16;
            mine = a.partial + ((static_cast<int64_t>(x.x) * (a.parts - 1) / a.parts + row - each * C) * p.Hv + h) * 2 * K;
        }
    }
    const bool in[2] = {row + g < own.y, row + g + 8 < own.y};
    if (mine) {                                            // the part's own outputs to L2
#pragma unroll
        for (int x = lane; x < 16 * (K / 32); x += 32) {
            const int r = x / (K / 32);
            if (row + r < own.y) asm volatile("prefetch.global.L2 [%0];" :: "l"(mine + r * ld + x % (K / 32) * 32));
        }
    }
    // the rows of the transition, all on their way beside the state
#pragma unroll
    for (int x = lane; x < 16 * (K / 4); x += 32) {
        const int r = x / (K / 4), c = x % (K / 4) * 4;
        const bool is = row + r < own.y;
        cp_async16(tc::smem_addr(rows + r * ROW + c), is ? mine + r * ld + K + c : a.partial, is);
    }
    cp_async_commit();
#pragma unroll 1
    for (int i = 0; i < 2; i++) {
        if (!from[i] || (i == 1 && from[1] == from[0])) continue;
        __syncthreads();
        if (tid < K) units[tid] = unit[i][tid];
        __syncthreads();
#pragma unroll 4
        for (int x = tid; x < K * K / 8; x += 256) {
            const int j = x / (K / 4), c = x % (K / 4) * 4;
            const float4 f0 = *reinterpret_cast<const float4 *>(from[i] + 2 * j * K + c), f1 = *reinterpret_cast<const float4 *>(from[i] + (2 * j + 1) * K + c);
            const float4 z = *reinterpret_cast<const float4 *>(units + c);
            const float4 r = make_float4(over(z.x), over(z.y), over(z.z), over(z.w));
            const uint4 y = make_uint4(tc::pack_f16x2(f0.x * r.x, f1.x * r.x), tc::pack_f16x2(f0.y * r.y, f1.y * r.y), tc::pack_f16x2(f0.z * r.z, f1.z * r.z),
                                       tc::pack_f16x2(f0.w * r.w, f1.w * r.w));
            *reinterpret_cast<uint4 *>(state + j * LD + c) = j & 2 ? make_uint4(y.z, y.w, y.x, y.y) : y;
        }
        __syncthreads();
        if (from[warp / 4] != from[i]) continue;
        // Of 16 of the inner axis a lane has columns 4 t .. 4 t + 3, which count as k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9; so too with the outputs' columns.
        auto four = [&](int r, int k) { return *reinterpret_cast<const float4 *>(rows + (g + 8 * r) * ROW + 16 * k + 4 * t); };
        cp_async_wait_all();
        __syncwarp();
        float whole[2] = {}, part[2];                      // the units of rows g and g + 8, and one over them
#pragma unroll
        for (int r = 0; r < 2; r++) {
#pragma unroll
            for (int k = 0; k < K / 16; k++) {
                const float4 x = four(r, k);
                whole[r] = fmaxf(fmaxf(whole[r], fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) whole[r] = fmaxf(whole[r], __shfl_xor_sync(0xffffffffu, whole[r], x));
            whole[r] = unit_of(whole[r]);
            part[r] = over(whole[r]);
        }
        float o[K / 8][4] = {};
#pragma unroll 2
        for (int k = 0; k < K / 16; k++) {
            uint32_t f[4];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float4 x = four(r, k);
                f[r] = tc::pack_f16x2(x.x * part[r], x.y * part[r]);
                f[2 + r] = tc::pack_f16x2(x.z * part[r], x.w * part[r]);
            }
            const uint32_t *s = state + (8 * k + 2 * t) * LD + (((g >> 1) * 4 + (g & 1)) ^ (t & 1) * 2);
#pragma unroll
            for (int n = 0; n < K / 8; n++) {
                const uint32_t *at = n % 2 ? s + 8 * n - 8 + (t & 1 ? -2 : 2) : s + 8 * n;
                mma_f16(o[n], f, at[0], at[LD]);
            }
        }
        const float *add = mine + g * ld + 4 * t;
        uint16_t *out = p.out + (static_cast<int64_t>(own.x) + row + g) * p.ld_out + static_cast<int64_t>(h) * K + 4 * t;
#pragma unroll
        for (int n = 0; n < K / 8; n += 2) {
            const float4 z = *reinterpret_cast<const float4 *>(units + 8 * n + 4 * t);
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float4 x = in[r] ? *reinterpret_cast<const float4 *>(add + 8 * r * ld + 8 * n) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float y[4] = {fmaf(o[n][2 * r] * whole[r], z.x, x.x), fmaf(o[n][2 * r + 1] * whole[r], z.y, x.y),
                                    fmaf(o[n + 1][2 * r] * whole[r], z.z, x.z), fmaf(o[n + 1][2 * r + 1] * whole[r], z.w, x.w)};
                if (in[r]) *reinterpret_cast<uint2 *>(out + 8 * r * p.ld_out + 8 * n) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            }
        }
    }
    cp_async_wait_all();                                   // a warp without a state to multiply has copies too
}

// ---- host ---------------------------------------------------------------------------------

// Shared memory of ends_kernel.
constexpr int ends_bytes(int K) { return (K * 32 + 2 * K * K + 8 * 32) * 4; }
// And of outputs_kernel.
constexpr int outputs_bytes(int K) { return (K / 2 * (K + 4) + 128 * (K + 16)) * 4; }

// The parts of long sequences: as many as give every chain a multiprocessor of a GB300's 152, with two chains for each part behind the first.
// (Not by the current device's: the workspace's size goes by the parts, and may be asked for where another device is current, or none.)
// Sequences that cannot have CUT_CHUNKS chunks on average stay whole: the joining costs 20 us and more. One sequence of K = V = 128, in parts and whole:
// 2048 tokens x 32 heads 111 and 107 us, 4096 x 32 188 and 202, 16,384 x 32 619 and 757, 4096 x 8 112 and 180, 16,384 x 8 239 and 682.
int parts_of(int64_t rows, int64_t num_seqs, int Hv, int K, int V)
{
    const int64_t chains = num_seqs * Hv;
    if (K != V || rows / num_seqs < CUT_CHUNKS * C) return 1;
    int64_t parts = (152 / chains + 1) / 2;
    if (parts > MOST_PARTS) parts = MOST_PARTS;
    return parts < 2 ? 1 : static_cast<int>(parts);
}

// Boxes of 64 rows by `box` columns of the packed q | k | v rows.
cudaError_t encode(CUtensorMap *m, const GdnParams &p, int64_t rows, int64_t cols, int box, CUtensorMapSwizzle swizzle)
{
    return mma::encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.qkv, cols, rows, p.ld_qkv, box, C, swizzle);
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
            const auto limit = [&](auto kernel, int bytes) {
                if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            };
            e = cudaDeviceGetAttribute(&counts[dev], cudaDevAttrMultiProcessorCount, dev);
            limit(prep_kernel<1>, HALF); limit(prep_kernel<2>, 2 * HALF);
            limit(ends_kernel<64>, ends_bytes(64)); limit(ends_kernel<128>, ends_bytes(128)); limit(outputs_kernel<64>, outputs_bytes(64)); limit(outputs_kernel<128>, outputs_bytes(128));
            limit(chain_kernel<1, 32, false>, Smem::END); limit(chain_kernel<1, 64, false>, Smem::END); limit(chain_kernel<1, 128, false>, Smem::END);
            limit(chain_kernel<2, 32, false>, Smem::END); limit(chain_kernel<2, 64, false>, Smem::END); limit(chain_kernel<2, 128, false>, Smem::END);
            limit(chain_kernel<1, 64, true>, Smem::END); limit(chain_kernel<2, 128, true>, Smem::END);
            if (e != cudaSuccess) return e;
            known[dev].store(true, std::memory_order_release);
        }
    }
    *sms = counts[dev];
    return cudaSuccess;
}

int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace
}  // namespace gdn

namespace gdn {
namespace {
// Where a call's arrays begin in its workspace.
struct Layout {
    int parts;
    int64_t where, records, states, units, partial, end;
    Layout(int64_t rows, int64_t num_seqs, int Hv, int K, int V) : parts(parts_of(rows, num_seqs, Hv, K, V))
    {
        const int64_t chunks = rows / C + num_seqs;
        where = up((num_seqs + 1) * 4);
        records = where + up(chunks * 8);
        states = records + up(chunks * Hv * Rec::BYTES);
        units = states + (parts > 1 ? num_seqs * Hv * (2 * parts - 1) * K * V * 4 : 0);
        partial = units + (parts > 1 ? num_seqs * Hv * (2 * parts - 1) * V * 4 : 0);
        end = partial + (parts > 1 ? rows * (parts - 1) / parts * Hv * (V + K) * 4 : 0);
    }
};
}  // namespace
}  // namespace gdn

size_t gdn_prefill_workspace(int64_t rows, int64_t num_seqs, int Hv, int K, int V)
{
    if (K == 32 || rows == 0 || num_seqs == 0) return 0;
    return static_cast<size_t>(gdn::Layout(rows, num_seqs, Hv, K, V).end);
}

cudaError_t launch_gdn_prefill(const GdnParams &p, int K, int V, const int32_t *cu, int64_t rows, int64_t num_seqs, void *workspace,
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
    const int64_t cols = 2 * static_cast<int64_t>(p.Hk) * K + static_cast<int64_t>(p.Hv) * V, chains = num_seqs * p.Hv;
    const Layout at(rows, num_seqs, p.Hv, K, V);
    // few chains: halves of their value columns, if there are idle multiprocessors for them (16,384 tokens x 32 heads in one part 779 us, whole columns 818,
    // quarters 812: the warps of the columns that are left use as many of the multiprocessor's quarters fewer, each as loaded as before)
    const int VS = V == 128 && at.parts == 1 && chains * 2 <= sms ? 64 : V;
    if ((e = encode(&qk, p, rows, cols, 64, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    if ((e = encode(&v, p, rows, cols, VS, CU_TENSOR_MAP_SWIZZLE_NONE)) != cudaSuccess) return e;
    const int64_t chunks = rows / C + num_seqs;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    const Args a{p, cu, static_cast<int>(rows), static_cast<int>(num_seqs), V, static_cast<int>(chunks), reinterpret_cast<int32_t *>(w),
                 reinterpret_cast<int2 *>(w + at.where), w + at.records, at.parts, reinterpret_cast<float *>(w + at.states),
                 reinterpret_cast<float *>(w + at.units), reinterpret_cast<float *>(w + at.partial)};
    if ((e = launch_pdl(map_kernel, dim3(1), dim3(1024), 0, stream, a)) != cudaSuccess) return e;
    const dim3 units(static_cast<unsigned>(chunks * p.Hk));
    e = K == 64 ? launch_pdl(prep_kernel<1>, units, dim3(128), HALF, stream, qk, a) : launch_pdl(prep_kernel<2>, units, dim3(128), 2 * HALF, stream, qk, a);
    if (e != cudaSuccess) return e;
    const int64_t ctas = chains * (V / VS) * (2 * at.parts - 1);
    const dim3 grid(static_cast<unsigned>(ctas < sms ? ctas : sms));
#define KDA_GDN_RUN(NH, W, PARTS) \
    if (K == 64 * NH && VS == W && (at.parts > 1) == PARTS) e = launch_pdl(chain_kernel<NH, W, PARTS>, grid, dim3(THREADS), Smem::END, stream, qk, v, a);
    KDA_GDN_RUN(1, 32, false) KDA_GDN_RUN(1, 64, false) KDA_GDN_RUN(1, 128, false) KDA_GDN_RUN(2, 32, false) KDA_GDN_RUN(2, 64, false)
    KDA_GDN_RUN(2, 128, false) KDA_GDN_RUN(1, 64, true) KDA_GDN_RUN(2, 128, true)
#undef KDA_GDN_RUN
    if (e != cudaSuccess || at.parts == 1) return e;
    const dim3 slices(static_cast<unsigned>(chains * (V / 32)));
    e = K == 64 ? launch_pdl(ends_kernel<64>, slices, dim3(256), ends_bytes(K), stream, a) : launch_pdl(ends_kernel<128>, slices, dim3(256), ends_bytes(K), stream, a);
    if (e != cudaSuccess) return e;
    const dim3 pairs(static_cast<unsigned>((chunks + 1) / 2 * p.Hv));
    return K == 64 ? launch_pdl(outputs_kernel<64>, pairs, dim3(256), outputs_bytes(64), stream, a) : launch_pdl(outputs_kernel<128>, pairs, dim3(256), outputs_bytes(128), stream, a);
}

}  // namespace kda
