// extern "C" entry points of the operators around the recurrence: host-side argument
// checks, then one launch on the caller's stream.
#include <climits>
#include <cmath>

#include "kda.h"
#include "kda_launch.h"
#include "kda_layer.h"

namespace {

using kda::set_error;

int done(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? set_error(KDA_OK, "%s", "") : set_error(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int invalid(const char *msg) { return set_error(KDA_ERR_INVALID_ARGUMENT, "%s", msg); }

int check_dtype(int32_t dtype, const char *name)
{
    if (dtype < KDA_BF16 || dtype > KDA_FP32)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "%s must be KDA_BF16, KDA_FP16 or KDA_FP32 (got %d)", name, dtype);
    return KDA_OK;
}

constexpr int64_t kMostSide = int64_t(1) << 30;   // of a product: tile ends past a side stay below 2^31

int fp8_matmul(const uint8_t *a, int64_t ld_a, const float *a_scales, int64_t sa_row_stride,
               int64_t sa_group_stride, const uint8_t *w, int64_t ld_w, const float *w_scales,
               int64_t sw_row_stride, int64_t sw_group_stride, int64_t M, int64_t N, int64_t K,
               void *out, int64_t ld_out, int32_t out_dtype, uint32_t *err_flags, int stalled, void *stream)
{
    int s;
    if ((s = check_dtype(out_dtype, "out_dtype"))) return s;
    if (M < 0 || N < 0 || K < 0 || M > kMostSide || N > kMostSide || K > kMostSide) return invalid("M, N and K must be in [0, 2^30]");
    if ((M + 63) / 64 * ((N + 63) / 64) > INT32_MAX)
        return set_error(KDA_ERR_UNSUPPORTED, "%lld x %lld outputs exceed one launch: split the call", (long long)M, (long long)N);
    if (M == 0 || N == 0) return set_error(KDA_OK, "%s", "");
    if (!out) return invalid("out must be non-NULL");
    if (K > 0 && (!a || !a_scales || !w || !w_scales)) return invalid("a, w and their scales must be non-NULL");
    if (ld_a < K || ld_w < K || ld_out < N) return invalid("row strides must be >= K (a, w) and >= N (out)");
    if (sa_row_stride < 1 || sa_group_stride < 1 || sw_row_stride < 1 || sw_group_stride < 1)
        return invalid("scale strides must be >= 1");
    if (!aligned(out, out_dtype == KDA_FP32 ? 4 : 2) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(err_flags, 4))
        return invalid("a pointer is not aligned to its element type");
    kda::Fp8Params p{a, ld_a, a_scales, sa_row_stride, sa_group_stride, w, ld_w, w_scales, sw_row_stride,
                 sw_group_stride, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), out, ld_out,
                 out_dtype, err_flags, stalled};
    return done(kda::launch_fp8_matmul(p, static_cast<cudaStream_t>(stream)), "kda_fp8_matmul launch");
}

}  // namespace

extern "C" {

int kda_norm_quant(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int32_t dtype,
                   const float *weight, float eps, int64_t N, int64_t D, void *residual_out,
                   int64_t ld_residual_out, void *y_out, int64_t ld_y, uint8_t *q, int64_t ld_q,
                   float *scales, int64_t scale_row_stride, int64_t scale_group_stride, void *stream)
{
    int s;
    if ((s = check_dtype(dtype, "dtype"))) return s;
    if (N < 0 || D < 1) return invalid("N must be >= 0 and D >= 1");
    if (D > kda::kNormMaxCols)
        return set_error(KDA_ERR_UNSUPPORTED, "D must be <= %d (got %lld)", kda::kNormMaxCols, (long long)D);
    if (N > INT32_MAX) return set_error(KDA_ERR_UNSUPPORTED, "N must be < 2^31: split the call");
    if (N == 0) return set_error(KDA_OK, "%s", "");
    if (!x || !q || !scales) return invalid("x, q and scales must be non-NULL");
    if (!residual != !residual_out) return invalid("residual and residual_out go together");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return invalid("eps must be finite and >= 0");
    if (ld_x < D || (residual && (ld_residual < D || ld_residual_out < D)) || (y_out && ld_y < D) || ld_q < D)
        return invalid("every row stride must be >= D");
    if (scale_row_stride < 1 || scale_group_stride < 1) return invalid("scale strides must be >= 1");
    const size_t es = dtype == KDA_FP32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(residual_out, es) || !aligned(y_out, es) ||
        !aligned(weight, 4) || !aligned(scales, 4))
        return invalid("a pointer is not aligned to its element type");
    kda::NormQuantParams p{x, ld_x, residual, ld_residual, weight, eps, residual_out, ld_residual_out, y_out, ld_y,
                           q, ld_q, scales, scale_row_stride, scale_group_stride, N, static_cast<int>(D)};
    return done(kda::launch_norm_quant(p, dtype, static_cast<cudaStream_t>(stream)), "kda_norm_quant launch");
}

int kda_fp8_matmul(const uint8_t *a, int64_t ld_a, const float *a_scales, int64_t sa_row_stride,
                   int64_t sa_group_stride, const uint8_t *w, int64_t ld_w, const float *w_scales,
                   int64_t sw_row_stride, int64_t sw_group_stride, int64_t M, int64_t N, int64_t K,
                   void *out, int64_t ld_out, int32_t out_dtype, uint32_t *err_flags, void *stream)
{
    return fp8_matmul(a, ld_a, a_scales, sa_row_stride, sa_group_stride, w, ld_w, w_scales, sw_row_stride, sw_group_stride, M, N, K, out,
                      ld_out, out_dtype, err_flags, -1, stream);
}

int kda_fp8_matmul_plan(const uint8_t *a, int64_t ld_a, const uint8_t *w, int64_t ld_w, int64_t M, int64_t N,
                        int64_t K, int32_t *plan)
{
    if (!plan) return invalid("plan must be non-NULL");
    if (M < 1 || N < 1 || K < 0 || M > kMostSide || N > kMostSide || K > kMostSide) return invalid("M and N must be in [1, 2^30], K in [0, 2^30]");
    if (ld_a < K || ld_w < K) return invalid("row strides must be >= K");
    kda::Fp8Params p{};
    p.a = a;
    p.ld_a = ld_a;
    p.w = w;
    p.ld_w = ld_w;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    int32_t got[3];
    const cudaError_t e = kda::plan_fp8_matmul(p, got);
    for (int i = 0; i < 3 && e == cudaSuccess; i++) plan[i] = got[i];
    return done(e, "kda_fp8_matmul_plan");
}

int kda_selftest_fp8_matmul(const uint8_t *a, int64_t ld_a, const float *a_scales, int64_t sa_row_stride,
                            int64_t sa_group_stride, const uint8_t *w, int64_t ld_w, const float *w_scales,
                            int64_t sw_row_stride, int64_t sw_group_stride, int64_t M, int64_t N, int64_t K,
                            void *out, int64_t ld_out, int32_t out_dtype, int32_t stalled, uint32_t *err_flags,
                            void *stream)
{
    if (!err_flags) return invalid("err_flags must be non-NULL");
    if (stalled < 0 || stalled > 7) return invalid("stalled must be in [0, 7]");
    return fp8_matmul(a, ld_a, a_scales, sa_row_stride, sa_group_stride, w, ld_w, w_scales, sw_row_stride, sw_group_stride, M, N, K, out,
                      ld_out, out_dtype, err_flags, stalled, stream);
}

int kda_batch_maps(const int32_t *query_lens, const int32_t *context_lens, const int32_t *state_slots,
                   int64_t state_stride, int64_t R, int32_t *block_table, int64_t table_stride,
                   int64_t table_width, const int32_t *free_pages, int64_t num_free,
                   const int32_t *free_count, int64_t num_pages, int32_t page_size, int64_t num_tokens,
                   int32_t *order, int32_t *cu_seqlens, int32_t *state_indices, int32_t *num_decodes,
                   int32_t *positions, int64_t *slot_map, int32_t *free_left, uint32_t *err_flags,
                   void *stream)
{
    if (R < 0 || num_tokens < 0 || num_free < 0 || num_pages < 0 || table_width < 0)
        return invalid("R, num_tokens, num_free, num_pages and table_width must be >= 0");
    if (R > (1 << 24) || num_tokens > INT32_MAX)
        return set_error(KDA_ERR_UNSUPPORTED, "R must be <= 2^24 and num_tokens < 2^31");
    if (num_free > INT32_MAX || num_pages > INT32_MAX || table_width > INT32_MAX)
        return invalid("num_free, num_pages and table_width must be < 2^31");
    if (page_size < 1) return invalid("page_size must be >= 1");
    if (!cu_seqlens || !num_decodes || !free_left || !free_count)
        return invalid("cu_seqlens, num_decodes, free_count and free_left must be non-NULL");
    if (R > 0 && (!query_lens || !context_lens || !state_slots || !order || !state_indices))
        return invalid("query_lens, context_lens, state_slots, order and state_indices must be non-NULL");
    if (R > 0 && table_width > 0 && (!block_table || table_stride < table_width))
        return invalid("block_table must be non-NULL with table_stride >= table_width");
    if (state_stride < 1) return invalid("state_stride must be >= 1");
    if (num_free > 0 && !free_pages) return invalid("free_pages must be non-NULL");
    if (num_tokens > 0 && (!positions || !slot_map)) return invalid("positions and slot_map must be non-NULL");
    if (free_left == free_count) return invalid("free_left must not be free_count");
    if (!aligned(query_lens, 4) || !aligned(context_lens, 4) || !aligned(state_slots, 4) || !aligned(block_table, 4) ||
        !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(order, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(state_indices, 4) || !aligned(num_decodes, 4) || !aligned(positions, 4) || !aligned(slot_map, 8) ||
        !aligned(free_left, 4) || !aligned(err_flags, 4))
        return invalid("a pointer is not aligned to its element type");
    kda::BatchMapsParams p{query_lens, context_lens, state_slots, state_stride, static_cast<int>(R), block_table,
                           table_stride, table_width, free_pages, num_free, free_count, num_pages, page_size,
                           num_tokens, order, cu_seqlens, state_indices, num_decodes, positions, slot_map,
                           free_left, err_flags};
    return done(kda::launch_batch_maps(p, static_cast<cudaStream_t>(stream)), "kda_batch_maps launch");
}

}  // extern "C"
