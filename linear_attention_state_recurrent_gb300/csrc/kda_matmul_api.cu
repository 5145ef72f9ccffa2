// extern "C" entry points of the 16-bit matrix product: host-side argument checks, then one launch on the caller's stream.
#include <climits>

#include "kda.h"
#include "kda_launch.h"
#include "kda_matmul.h"

namespace {

using kda::set_error;

int invalid(const char *msg) { return set_error(KDA_ERR_INVALID_ARGUMENT, "%s", msg); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t size_of(int32_t dtype) { return dtype == KDA_FP32 ? 4 : 2; }

int done(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? set_error(KDA_OK, "%s", "") : set_error(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int64_t kMostSide = int64_t(1) << 30;   // tile ends past a side stay below 2^31

}  // namespace

extern "C" {

int kda_matmul(const void *a, int64_t ld_a, const void *w, int64_t ld_w, int32_t dtype, int64_t M, int64_t N, int64_t K, const void *bias,
               int32_t bias_dtype, int32_t act, const void *residual, int64_t ld_residual, void *out, int64_t ld_out, int32_t out_dtype,
               uint32_t *err_flags, void *stream)
{
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return set_error(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_BF16 or KDA_FP16 (got %d)", dtype);
    if (out_dtype < KDA_BF16 || out_dtype > KDA_FP32)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "out_dtype must be KDA_BF16, KDA_FP16 or KDA_FP32 (got %d)", out_dtype);
    if (bias && bias_dtype != dtype && bias_dtype != KDA_FP32) return invalid("bias_dtype must be dtype or KDA_FP32");
    if (act < KDA_ACT_NONE || act > KDA_ACT_GELU_TANH) return set_error(KDA_ERR_INVALID_ARGUMENT, "act must be a KDA_ACT_* (got %d)", act);
    if (M < 0 || N < 0 || K < 0 || M > kMostSide || N > kMostSide || K > kMostSide) return invalid("M, N and K must be in [0, 2^30]");
    if ((M + 63) / 64 * ((N + 127) / 128) > INT32_MAX / 8)   // tiles of the slowest arrangement, split eight ways
        return set_error(KDA_ERR_UNSUPPORTED, "%lld x %lld outputs exceed one launch: split the call", (long long)M, (long long)N);
    if (M == 0 || N == 0) return set_error(KDA_OK, "%s", "");
    if (!out) return invalid("out must be non-NULL");
    if (K > 0 && (!a || !w)) return invalid("a and w must be non-NULL");
    if (ld_a < K || ld_w < K || ld_out < N || (residual && ld_residual < N)) return invalid("row strides must be >= K (a, w) and >= N (out, residual)");
    if (!aligned(a, 2) || !aligned(w, 2) || !aligned(out, size_of(out_dtype)) || !aligned(residual, size_of(out_dtype)) ||
        (bias && !aligned(bias, size_of(bias_dtype))) || !aligned(err_flags, 4))
        return invalid("a pointer is not aligned to its element type");
    const kda::MatmulParams p{a, ld_a, w, ld_w, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), bias, bias_dtype, act, residual,
                              ld_residual, out, ld_out, dtype, out_dtype, err_flags};
    const cudaError_t e = kda::launch_matmul(p, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration)
        return set_error(KDA_ERR_UNSUPPORTED, "%lld x %lld outputs of these operands exceed one launch: split the call", (long long)M, (long long)N);
    return done(e, "kda_matmul launch");
}

int kda_matmul_plan(const void *a, int64_t ld_a, const void *w, int64_t ld_w, int64_t M, int64_t N, int64_t K, int32_t *plan)
{
    if (!plan) return invalid("plan must be non-NULL");
    if (M < 1 || N < 1 || K < 0 || M > kMostSide || N > kMostSide || K > kMostSide) return invalid("M and N must be in [1, 2^30], K in [0, 2^30]");
    if (ld_a < K || ld_w < K) return invalid("row strides must be >= K");
    kda::MatmulParams p{};
    p.a = a;
    p.ld_a = ld_a;
    p.w = w;
    p.ld_w = ld_w;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    int32_t got[2];
    const cudaError_t e = kda::plan_matmul(p, got);
    for (int i = 0; i < 2 && e == cudaSuccess; i++) plan[i] = got[i];
    return done(e, "kda_matmul_plan");
}

}  // extern "C"
