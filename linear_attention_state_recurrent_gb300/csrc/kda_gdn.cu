// The gated delta rule with one decay per token and head, token by token or in blocks of a few tokens.
//
//   S <- alpha S,  u = beta (v - S^T k^),  S <- S + k^ u^T,  o = S^T q^       (S fp32 [K][V] per value head)
//
// with alpha = exp(-e^{A_log} softplus(raw_g + dt_bias)) and value head h on key head h / (Hv / Hk).
//
// decode_kernel: one token. A CTA owns a slice of 32 value columns of one state (they are independent: column j of
// the new S depends on column j of the old one alone). Bound by the state's bytes.
//
// rows_kernel: n tokens per step, n <= 8 or 16, on mma.sync, for the requests of a few rows and for what the chunked
// kernel does not take (K = 32, rows off 16-byte boundaries). With b the running log-decay inside the block, D[r, i] = e^{b_r - b_i},
// A[r, i] = beta_r (k^_r . k^_i) D[r, i] (i < r) and T = (I + A)^-1, the block's tokens need S only twice:
//   U = T diag(beta) (v - e^b (k^ S)),  o = e^b (q^ S) + (q^ k^^T * D) U,  S <- e^{b_n} S + (k^ e^{b_n - b})^T U
// so a state is read from memory once, kept in registers as the MMAs' accumulators, and written once. It is held
// transposed (rows of an MMA = value columns, columns = key channels): the accumulator layout is then the layout of the
// first operand of the next product. fp32 values enter the MMAs as two tf32 terms (2^-20 of the value); q and k are bf16, exact in one. (With
// two bf16 terms, 2^-17, the states were off by 2e-6 to 6e-6 of their norm, for 20.4 us instead of 21.4 at 16 x 8 rows x 32 heads.)
#include "kda_gdn_common.cuh"
#include "kda_pdl.cuh"

namespace kda {
namespace gdn {

template <int K, int V>
__global__ void __launch_bounds__(128, 12) decode_kernel(GdnParams p)
{
    constexpr int VT = 32, VS = V / VT, RPT = K / 16, CPL = K / 32;
    // Thread (rg, cg) copies, reads and stores rows rg, rg + 16, .. of four columns: no register holds the slice, and
    // shared memory (17.9 KB at K = 128) lets twelve CTAs have their loads in flight on an SM.
    __shared__ __align__(16) float4 s_tile[RPT][128];
    __shared__ uint32_t s_kq[K];                           // bf16 k | q << 16
    __shared__ __align__(16) float4 s_red[4][2][VT / 4];   // [warp][k^T S, q^T S][column group]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cg = tid & 7, rg = tid >> 3;
    pdl_wait_then_release();   // no global read before this

    const int64_t b = blockIdx.x;
    const int vs = static_cast<int>(b % VS);
    const int h = static_cast<int>((b / VS) % p.Hv), hk = h / (p.Hv / p.Hk);
    const int64_t e = b / (static_cast<int64_t>(VS) * p.Hv);
    const int j0 = vs * VT + cg * 4;
    const int64_t slot = load_slot(p, e);
    uint16_t *orow = p.out + e * p.ld_out + static_cast<int64_t>(h) * V + j0;
    if (slot >= p.num_slots) {                             // out of range: flag, zero outputs
        if (tid == 0 && p.err) atomicOr(p.err, kErrSlotRange);
        if (rg == 0) *reinterpret_cast<uint2 *>(orow) = make_uint2(0u, 0u);
        return;
    }
    const bool has_state = slot >= 0, writable = has_state && slot != p.null_slot;
    float *tile = has_state ? p.pool + slot * p.slot_stride + static_cast<int64_t>(h) * K * V + j0 : nullptr;
    if (has_state) {
#pragma unroll
        for (int i = 0; i < RPT; i++)
            cp_async16(static_cast<uint32_t>(__cvta_generic_to_shared(&s_tile[i][tid])), tile + static_cast<int64_t>(rg + 16 * i) * V, true);
    }
    cp_async_commit();

    const int64_t HK = static_cast<int64_t>(p.Hk) * K;
    const uint16_t *row = p.qkv + e * p.ld_qkv;
    uint16_t qb[CPL], kb[CPL];
#pragma unroll
    for (int c = 0; c < CPL; c++) {
        qb[c] = row[hk * K + lane + 32 * c];
        kb[c] = row[HK + hk * K + lane + 32 * c];
    }
    const uint16_t *vp = row + 2 * HK + static_cast<int64_t>(h) * V + j0;
    const float vv[4] = {bf16_to_f32(vp[0]), bf16_to_f32(vp[1]), bf16_to_f32(vp[2]), bf16_to_f32(vp[3])};
    const float beta = sigmoid_f(bf16_to_f32(p.rb[e * p.ld_beta + h]));
    const float alpha = expf(log_decay(p.rg[e * p.ld_g + h], expf(p.A_log[h]), p.dt_bias ? p.dt_bias[h] : 0.f));
    if (tid < K) {
        uint32_t kq = 0;
#pragma unroll
        for (int c = 0; c < CPL; c++)
            if (c == warp) kq = static_cast<uint32_t>(kb[c]) | (static_cast<uint32_t>(qb[c]) << 16);
        s_kq[tid] = kq;
    }
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; c++) {
        const float qf = bf16_to_f32(qb[c]), kf = bf16_to_f32(kb[c]);
        qq += qf * qf; kk += kf * kf; qk += qf * kf;
    }
    qq = warp_sum(qq);
    kk = warp_sum(kk);
    qk = warp_sum(qk);
    cp_async_wait_all();   // this thread's own copies
    __syncthreads();

    const float rq = p.scale * rsqrtf(qq + p.eps), rk = rsqrtf(kk + p.eps);
    float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RPT; i++) {
        const uint32_t kq = s_kq[rg + 16 * i];
        const float kr = __uint_as_float(kq << 16), qr = __uint_as_float(kq & 0xffff0000u);
        const float4 S = has_state ? s_tile[i][tid] : make_float4(0.f, 0.f, 0.f, 0.f);
        pk[0] += kr * S.x; pk[1] += kr * S.y; pk[2] += kr * S.z; pk[3] += kr * S.w;
        pq[0] += qr * S.x; pq[1] += qr * S.y; pq[2] += qr * S.z; pq[3] += qr * S.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; jj++) {
        pk[jj] += __shfl_xor_sync(0xffffffffu, pk[jj], 8);
        pk[jj] += __shfl_xor_sync(0xffffffffu, pk[jj], 16);
        pq[jj] += __shfl_xor_sync(0xffffffffu, pq[jj], 8);
        pq[jj] += __shfl_xor_sync(0xffffffffu, pq[jj], 16);
    }
    if (lane < 8) {
        s_red[warp][0][cg] = make_float4(pk[0], pk[1], pk[2], pk[3]);
        s_red[warp][1][cg] = make_float4(pq[0], pq[1], pq[2], pq[3]);
    }
    __syncthreads();

    float u[4], o[4];
    const float qkh = qk * rq * rk;
    {
        float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; w++) {
            const float4 kw = s_red[w][0][cg], qw = s_red[w][1][cg];
            ks[0] += kw.x; ks[1] += kw.y; ks[2] += kw.z; ks[3] += kw.w;
            qs[0] += qw.x; qs[1] += qw.y; qs[2] += qw.z; qs[3] += qw.w;
        }
#pragma unroll
        for (int jj = 0; jj < 4; jj++) {
            u[jj] = beta * (vv[jj] - alpha * (ks[jj] * rk));
            o[jj] = alpha * (qs[jj] * rq) + qkh * u[jj];
        }
    }
    if (rg == 0) *reinterpret_cast<uint2 *>(orow) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    if (writable) {
#pragma unroll
        for (int i = 0; i < RPT; i++) {
            const int r = rg + 16 * i;
            const float kh = __uint_as_float(s_kq[r] << 16) * rk;
            float4 S = s_tile[i][tid];
            S.x = fmaf(S.x, alpha, kh * u[0]); S.y = fmaf(S.y, alpha, kh * u[1]);
            S.z = fmaf(S.z, alpha, kh * u[2]); S.w = fmaf(S.w, alpha, kh * u[3]);
            *reinterpret_cast<float4 *>(tile + static_cast<int64_t>(r) * V) = S;
        }
    }
}

// ---- mma.sync ----------------------------------------------------------------------------

// d += a b, 16 rows by 8 columns, k = 16
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A tile of accumulators as the first operand of a product over its columns: column 2t counts as k = t, 2t + 1 as k = t + 4.
__device__ __forceinline__ Tf32<4> operand(const float (&x)[4])
{
    Tf32<4> r;
    r.set(0, x[0]); r.set(1, x[2]); r.set(2, x[1]); r.set(3, x[3]);
    return r;
}
// A pair of bf16 values (columns 2t, 2t + 1) as the second operand, exact.
__device__ __forceinline__ void mma_pair(float (&d)[4], const Tf32<4> &a, uint32_t pair)
{
    const uint32_t b[2] = {pair << 16, pair & 0xffff0000u};
    mma_tf32(d, a.lo, b);
    mma_tf32(d, a.hi, b);
}

// Four 8 x 8 bf16 tiles, transposed; lane l gives the address of row l % 8 of tile l / 8.
__device__ __forceinline__ void load_trans(uint32_t (&r)[4], uint32_t saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr));
}

__device__ __forceinline__ float sum_squares(uint32_t pair)
{
    const float x = __uint_as_float(pair << 16), y = __uint_as_float(pair & 0xffff0000u);
    return x * x + y * y;
}

// Whether one of a pair of bf16 values is an infinity or NaN.
__device__ __forceinline__ bool not_finite(uint32_t pair)
{
    return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}

// One CTA per (entry, value head, 64 value columns): a warp holds 16 of them, in registers over all K channels (K / 2 floats a
// thread), and needs nothing of the other warps but the block's T and the query-key products, which warps 0 and 1 form while the
// others already multiply. TB tokens a step (a multiple of 8). Bound by the latency of a CTA's load, products and store, one after the other, so
// by how many CTAs are on an SM: with 32 columns a warp (three CTAs of a whole head an SM) 16 requests of 8 rows x 32 heads took a tenth longer.
template <int V>
constexpr int COLS = V < 64 ? V : 64;
// GROUPS: 128 threads each that an SM has to hold (four of them at K = 128: 128 registers a thread, hardly a spill).
template <int K, int V, int TB, int GROUPS>
__global__ void __launch_bounds__(2 * COLS<V>, GROUPS * 128 / (2 * COLS<V>))
rows_kernel(GdnParams p, int T, const int32_t *cu, int64_t rows, int vec, int ahead)
{
    constexpr int NT = TB / 8, CT = K / 8, PITCH = K + 8, TP = TB + 8, THREADS = 2 * COLS<V>, SLICES = V / COLS<V>;
    __shared__ __align__(16) uint16_t s_k[TB][PITCH], s_q[TB][PITCH];
    __shared__ __align__(8) float s_t[TB][TP], s_w[TB][TP];   // T diag(beta) and the scaled q k^T
    __shared__ float s_a[TB][TB + 1];
    __shared__ float s_ys[TB], s_qs[TB], s_us[TB];        // scales of k S, q S, and of U on its way into S
    __shared__ float s_gamma;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
    pdl_wait_then_release();   // no global read before this
    const int64_t e = blockIdx.x / (SLICES * p.Hv);
    const int h = static_cast<int>(blockIdx.x / SLICES % p.Hv), hk = h / (p.Hv / p.Hk);
    const int j0 = static_cast<int>(blockIdx.x % SLICES) * COLS<V> + warp * 16 + g * 2;   // this thread's two value columns
    int64_t row0 = e * T, row1 = row0 + T;
    if (cu) {
        row0 = cu[e];
        row1 = cu[e + 1];
        if (row0 < 0 || row1 < row0 || row1 > rows) {     // not a range of the rows: counts as empty
            if (tid == 0 && p.err) atomicOr(p.err, kErrLengths);
            row1 = row0;
        }
    }
    const int64_t HK = static_cast<int64_t>(p.Hk) * K;
    const float rate = p.A_log[h], dtb = p.dt_bias ? p.dt_bias[h] : 0.f;
    // A block's inputs, asked for before anything is waited for: q and k, v of this thread's columns and tokens, and the gates, in the two
    // warps that use them (lane r has token r's). Rows past the block's end are zeros.
    constexpr int QK = 2 * TB * (K / 8), PER = (QK + THREADS - 1) / THREADS;
    int n;
    uint4 qk[PER];
    uint32_t vr[NT][2];
    uint16_t raw_g, raw_b;
    auto fetch = [&](int64_t r0) {
        const uint16_t *in = p.qkv + r0 * p.ld_qkv;
#pragma unroll
        for (int x = 0; x < PER; x++) {
            const int i = tid + x * THREADS, part = i / (TB * (K / 8)), r = i / (K / 8) % TB, c = i % (K / 8) * 8;
            qk[x] = make_uint4(0u, 0u, 0u, 0u);
            if (i < QK && r < n) {
                const uint16_t *from = in + r * p.ld_qkv + part * HK + hk * K + c;
                if (vec) {
                    qk[x] = *reinterpret_cast<const uint4 *>(from);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; y++) w[y] = from[2 * y] | static_cast<uint32_t>(from[2 * y + 1]) << 16;
                    qk[x] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < NT; m++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int r = 8 * m + t2 + c;
                vr[m][c] = 0u;
                if (r < n) {
                    const uint16_t *vp = in + r * p.ld_qkv + 2 * HK + static_cast<int64_t>(h) * V + j0;
                    vr[m][c] = vec ? *reinterpret_cast<const uint32_t *>(vp) : vp[0] | static_cast<uint32_t>(vp[1]) << 16;
                }
            }
        if (warp < 2 && lane < n) {
            raw_g = p.rg[(r0 + lane) * p.ld_g + h];
            raw_b = p.rb[(r0 + lane) * p.ld_beta + h];
        }
    };
    n = row1 - row0 < TB ? static_cast<int>(row1 - row0) : TB;
    fetch(row0);
    const int64_t slot = load_slot(p, e);
    uint16_t *out = p.out + static_cast<int64_t>(h) * V + j0;
    if (slot >= p.num_slots) {                            // out of range: flag, zero outputs
        if (tid == 0 && p.err) atomicOr(p.err, kErrSlotRange);
        for (int64_t r = row0 + (lane & 3); r < row1; r += 4) *reinterpret_cast<uint32_t *>(out + r * p.ld_out) = 0u;
        return;
    }
    if (row0 == row1) return;
    const bool has_state = slot >= 0, writable = has_state && slot != p.null_slot;
    float *tile = has_state ? p.pool + slot * p.slot_stride + static_cast<int64_t>(h) * K * V + j0 : nullptr;

    // S[n]: columns j0, j0 + 1 (the MMA's rows g and g + 8), channels 8n + t2, 8n + t2 + 1
    float S[CT][4];
#pragma unroll
    for (int i = 0; i < CT; i++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const float2 x = has_state ? *reinterpret_cast<const float2 *>(tile + static_cast<int64_t>(8 * i + t2 + c) * V) : make_float2(0.f, 0.f);
            S[i][c] = x.x; S[i][2 + c] = x.y;
        }

    // A block's products take zeros for the rows behind a row, and 0 times what is not finite is not 0: where a block's keys, values
    // or gates are not all finite, its rows go one by one, and those ahead of such a row stay as they are.
    for (int64_t r0 = row0;;) {
        float vv[NT][4], gl, beta;
#pragma unroll 1
        for (;;) {
            bool odd = false;
#pragma unroll
            for (int x = 0; x < PER; x++) {
                const int i = tid + x * THREADS, part = i / (TB * (K / 8)), r = i / (K / 8) % TB, c = i % (K / 8) * 8;
                if (i >= QK) break;
                odd |= part && (not_finite(qk[x].x) || not_finite(qk[x].y) || not_finite(qk[x].z) || not_finite(qk[x].w));
                *reinterpret_cast<uint4 *>(part ? &s_k[r][c] : &s_q[r][c]) = qk[x];
            }
#pragma unroll
            for (int m = 0; m < NT; m++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    odd |= not_finite(vr[m][c]);
                    vv[m][c] = __uint_as_float(vr[m][c] << 16); vv[m][2 + c] = __uint_as_float(vr[m][c] & 0xffff0000u);
                }
            gl = 0.f;
            beta = 0.f;
            if (warp < 2 && lane < n) {
                gl = log_decay(raw_g, expf(rate), dtb);
                beta = sigmoid_f(bf16_to_f32(raw_b));
                odd |= !(fabsf(gl) <= 1000.f && beta <= 1.f);
            }
            if (!__syncthreads_or(odd) || n == 1) break;
            n = 1;
            fetch(r0);
        }

        if (r0 == row0 && warp >= THREADS / 64) {
            // the state of the CTA that will follow this one on its multiprocessor, to L2
            const int64_t later = blockIdx.x + static_cast<int64_t>(ahead);
            const int64_t next = later < gridDim.x ? load_slot(p, later / (SLICES * p.Hv)) : -1;
            if (next >= 0 && next < p.num_slots) {
                const float *from = p.pool + next * p.slot_stride + (later / SLICES % p.Hv) * K * V + later % SLICES * COLS<V>;
                for (int i = tid - THREADS / 2; i < K * COLS<V> / 32; i += THREADS / 2)
                    asm volatile("prefetch.global.L2 [%0];" :: "l"(from + static_cast<int64_t>(i / (COLS<V> / 32)) * V + i % (COLS<V> / 32) * 32));
            }
        }
        // Warp 0: the block's scalars and T. Warp 1: the query-key products.
        if (warp < 2) {
            const RunningDecay b(gl, TB);
            const RunningDecay::At b_end = b.of(TB - 1);
            {
                const bool query = warp == 1;
                const uint16_t(*s_l)[PITCH] = query ? s_q : s_k;
                float G[NT][4] = {}, nl[2] = {}, nr[NT] = {};
#pragma unroll
                for (int kt = 0; kt < K / 16; kt++) {
                    uint32_t a[4] = {};
                    const int c = 16 * kt + t2;
                    a[0] = *reinterpret_cast<const uint32_t *>(&s_l[g][c]);
                    a[2] = *reinterpret_cast<const uint32_t *>(&s_l[g][c + 8]);
                    if (NT > 1) {
                        a[1] = *reinterpret_cast<const uint32_t *>(&s_l[(g + 8) % TB][c]);
                        a[3] = *reinterpret_cast<const uint32_t *>(&s_l[(g + 8) % TB][c + 8]);
                    }
                    nl[0] += sum_squares(a[0]) + sum_squares(a[2]);
                    nl[1] += sum_squares(a[1]) + sum_squares(a[3]);
#pragma unroll
                    for (int m = 0; m < NT; m++) {
                        uint32_t kb[2] = {*reinterpret_cast<const uint32_t *>(&s_k[8 * m + g][c]), *reinterpret_cast<const uint32_t *>(&s_k[8 * m + g][c + 8])};
                        nr[m] += sum_squares(kb[0]) + sum_squares(kb[1]);
                        mma(G[m], a, kb);
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    nl[0] += __shfl_xor_sync(0xffffffffu, nl[0], o);
                    nl[1] += __shfl_xor_sync(0xffffffffu, nl[1], o);
#pragma unroll
                    for (int m = 0; m < NT; m++) nr[m] += __shfl_xor_sync(0xffffffffu, nr[m], o);
                }
                // rows past the block's end have no norm: with eps = 0 theirs would be infinite
                nl[0] = g < n ? rsqrtf(nl[0] + p.eps) : 0.f;
                nl[1] = g + 8 < n ? rsqrtf(nl[1] + p.eps) : 0.f;
#pragma unroll
                for (int m = 0; m < NT; m++) nr[m] = rsqrtf(nr[m] + p.eps);
                // entry (r, i) of G: r = g + 8 hh, i = 8 m + t2 + c
#pragma unroll
                for (int hh = 0; hh < NT; hh++) {
                    const int r = g + 8 * hh;
                    const RunningDecay::At br = b.of(r);
                    const float beta_r = __shfl_sync(0xffffffffu, beta, r);
#pragma unroll
                    for (int m = 0; m < NT; m++)
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            const int i = 8 * m + t2 + c;
                            const RunningDecay::At bi = b.of(i);
                            const float ni = __shfl_sync(0xffffffffu, nr[m], (t2 + c) * 4);
                            const float x = G[m][2 * hh + c] * nl[hh] * ni;
                            if (!query) {
                                s_a[r][i] = i < r && r < n ? beta_r * x * expf(br - bi) : 0.f;
                            } else {
                                s_w[r][i] = i <= r && r < n ? p.scale * x * expf(br - bi) : 0.f;
                            }
                        }
                    if (t2 == 0) {
                        if (!query) {
                            s_ys[r] = expf(br) * nl[hh];
                            s_us[r] = expf(b_end - br) * nl[hh];
                        } else {
                            s_qs[r] = p.scale * expf(br) * nl[hh];
                        }
                    }
                }
                if (!query) {
                    if (lane == 0) s_gamma = expf(b_end);
                    __syncwarp();
                    // column `lane` of T by substitution, row after row
                    float x[TB];
#pragma unroll
                    for (int r = 0; r < TB; r++) {
                        float y = r == lane ? 1.f : 0.f;
#pragma unroll
                        for (int i = 0; i < r; i++) y = fmaf(-s_a[r][i], x[i], y);
                        x[r] = y;
                    }
                    if (lane < TB) {
#pragma unroll
                        for (int r = 0; r < TB; r++) s_t[r][lane] = x[r] * beta;
                    }
                }
            }
        }

        // k S and q S
        float P[NT][4] = {}, Q[NT][4] = {};
#pragma unroll
        for (int ct = 0; ct < CT; ct++) {
            const Tf32<4> x = operand(S[ct]);
#pragma unroll
            for (int r = 0; r < NT; r++) {
                mma_pair(P[r], x, *reinterpret_cast<const uint32_t *>(&s_k[8 * r + g][8 * ct + t2]));
                mma_pair(Q[r], x, *reinterpret_cast<const uint32_t *>(&s_q[8 * r + g][8 * ct + t2]));
            }
        }
        __syncthreads();   // T, the query-key products and the scales are there

        const float gamma = s_gamma;
        Tf32<4> x[NT];
        float U[NT][4] = {};
        // y = v - e^b (k^ S)
#pragma unroll
        for (int r = 0; r < NT; r++) {
            const float y0 = s_ys[8 * r + t2], y1 = s_ys[8 * r + t2 + 1];
            x[r] = operand({vv[r][0] - y0 * P[r][0], vv[r][1] - y1 * P[r][1], vv[r][2] - y0 * P[r][2], vv[r][3] - y1 * P[r][3]});
        }
        // d += x m^T, rows 8 r .. of m; tiles above the diagonal are zeros
        auto times = [&](float(&d)[4], const float(*m)[TP], int r) {
#pragma unroll
            for (int i = 0; i <= r; i++) {
                const float2 f = *reinterpret_cast<const float2 *>(&m[8 * r + g][8 * i + t2]);
                Tf32<2> b;
                b.set(0, f.x);
                b.set(1, f.y);
                mma_split(d, x[i], b);
            }
        };
#pragma unroll
        for (int r = 0; r < NT; r++) times(U[r], s_t, r);
        // o = e^b (q^ S) + W U
#pragma unroll
        for (int r = 0; r < NT; r++) x[r] = operand(U[r]);
#pragma unroll
        for (int r = 0; r < NT; r++) {
            const float q0 = s_qs[8 * r + t2], q1 = s_qs[8 * r + t2 + 1];
            Q[r][0] *= q0; Q[r][1] *= q1; Q[r][2] *= q0; Q[r][3] *= q1;
            times(Q[r], s_w, r);
        }
        // S <- gamma S + (k^ e^{b_n - b})^T U
#pragma unroll
        for (int r = 0; r < NT; r++) {
            const float u0 = s_us[8 * r + t2], u1 = s_us[8 * r + t2 + 1];
            x[r] = operand({U[r][0] * u0, U[r][1] * u1, U[r][2] * u0, U[r][3] * u1});
        }
#pragma unroll
        for (int ct = 0; ct < CT; ct += 4 / NT) {         // four 8 x 8 tiles of k: 4 / NT channel tiles of NT token tiles
            uint32_t kt[4];
            const int at = lane / 8;
            load_trans(kt, static_cast<uint32_t>(__cvta_generic_to_shared(&s_k[8 * (at % NT) + lane % 8][8 * (ct + at / NT)])));
#pragma unroll
            for (int c = 0; c < 4 / NT; c++) {
                float(&d)[4] = S[ct + c];
                d[0] *= gamma; d[1] *= gamma; d[2] *= gamma; d[3] *= gamma;
#pragma unroll
                for (int r = 0; r < NT; r++) mma_pair(d, x[r], kt[c * NT + r]);
            }
        }
#pragma unroll
        for (int r = 0; r < NT; r++)
#pragma unroll
            for (int c = 0; c < 2; c++)
                if (8 * r + t2 + c < n)
                    *reinterpret_cast<uint32_t *>(out + (r0 + 8 * r + t2 + c) * p.ld_out) = pack_bf16x2(Q[r][c], Q[r][2 + c]);
        r0 += n;
        if (r0 >= row1) break;
        n = row1 - r0 < TB ? static_cast<int>(row1 - r0) : TB;
        fetch(r0);
        __syncthreads();   // the block's q, k, T and scales have been read
    }
    if (writable) {
#pragma unroll
        for (int n = 0; n < CT; n++)
#pragma unroll
            for (int c = 0; c < 2; c++)
                *reinterpret_cast<float2 *>(tile + static_cast<int64_t>(8 * n + t2 + c) * V) = make_float2(S[n][c], S[n][2 + c]);
    }
}

}  // namespace gdn

#define KDA_GDN_DIMS(RUN) \
    RUN(32, 32) RUN(32, 64) RUN(32, 128) RUN(64, 32) RUN(64, 64) RUN(64, 128) RUN(128, 32) RUN(128, 64) RUN(128, 128)

cudaError_t launch_gdn_decode(const GdnParams &p, int K, int V, int64_t num_seqs, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(num_seqs * p.Hv * (V / 32)));
#define KDA_GDN_RUN(KK, VV) \
    if (K == KK && V == VV) return launch_pdl(gdn::decode_kernel<KK, VV>, grid, dim3(128), 0, stream, p);
    KDA_GDN_DIMS(KDA_GDN_RUN)
#undef KDA_GDN_RUN
    return cudaErrorInvalidValue;
}

cudaError_t launch_gdn_rows(const GdnParams &p, int K, int V, int T, const int32_t *cu, int64_t rows, int64_t num_entries,
                            cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(num_entries * p.Hv * (V > 64 ? V / 64 : 1)));
    const int vec = reinterpret_cast<uintptr_t>(p.qkv) % 16 == 0 && p.ld_qkv % 8 == 0;   // K and V are multiples of 8
    // Four groups of 128 threads an SM at K = 128, five where that saves a wave: 16 requests x 32 heads x 128 columns (1024 groups, two waves either way)
    // 18.9 us with four, 21.7 with five; 61 x 12 x 64 (732 groups) 15.5 with four, 13.7 with five.
    const int64_t groups = static_cast<int64_t>(grid.x) * (V < 64 ? V : 64) / 64;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const auto ahead = [&](int threads, int g) { return sms * (g * 128 / threads); };
    const bool five = (groups + 5 * sms - 1) / (5 * sms) < (groups + 4 * sms - 1) / (4 * sms);
    // blocks of 8 rows for requests of at most 8: half the products of 16
    const bool small = !cu && T <= 8;
#define KDA_GDN_LAUNCH(KK, VV, TB, G) return launch_pdl(gdn::rows_kernel<KK, VV, TB, G>, grid, dim3(2 * gdn::COLS<VV>), 0, stream, p, T, cu, rows, vec, ahead(2 * gdn::COLS<VV>, G));
#define KDA_GDN_RUN(KK, VV) \
    if (K == KK && V == VV) { \
        if (!small) KDA_GDN_LAUNCH(KK, VV, 16, KK == 128 ? 4 : 5) \
        if (five) KDA_GDN_LAUNCH(KK, VV, 8, KK == 128 ? 5 : 6) \
        KDA_GDN_LAUNCH(KK, VV, 8, KK == 128 ? 4 : 6) \
    }
    KDA_GDN_DIMS(KDA_GDN_RUN)
#undef KDA_GDN_RUN
#undef KDA_GDN_LAUNCH
    return cudaErrorInvalidValue;
}

}  // namespace kda
