// extern "C" entry points of the gated delta rule with one decay per head: host-side argument checks, then one launch
// on the caller's stream.
#include <climits>
#include <cmath>

#include "kda.h"
#include "kda_gdn.h"
#include "kda_launch.h"

namespace {

using kda::set_error;

int invalid(const char *msg) { return set_error(KDA_ERR_INVALID_ARGUMENT, "%s", msg); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_dim(int d) { return d == 32 || d == 64 || d == 128; }

// The checks that all calls share; fills the kernels' parameters.
int check(const uint16_t *mixed_qkv, int64_t ld_qkv, const uint16_t *raw_g, int64_t ld_g, const uint16_t *raw_beta,
          int64_t ld_beta, int64_t entries, const kda_gdn_heads *hd, const kda_state *st, uint16_t *out, int64_t ld_out,
          uint32_t *err_flags, kda::GdnParams *p)
{
    if (!hd) return invalid("heads is NULL");
    if (hd->Hk < 1 || hd->Hv < 1 || hd->Hv % hd->Hk != 0)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "Hk must be >= 1 and Hv a multiple of it (got %d, %d)", hd->Hk, hd->Hv);
    if (!supported_dim(hd->K) || !supported_dim(hd->V))
        return set_error(KDA_ERR_UNSUPPORTED, "K and V must each be 32, 64 or 128 (got K=%d, V=%d)", hd->K, hd->V);
    if (!hd->A_log) return invalid("A_log is NULL");
    if (!std::isfinite(hd->scale)) return invalid("scale must be finite");
    if (!(hd->l2_eps >= 0.f) || !std::isfinite(hd->l2_eps)) return invalid("l2_eps must be finite and >= 0");
    const int64_t Hk = hd->Hk, Hv = hd->Hv, K = hd->K, V = hd->V;
    if (!mixed_qkv || !raw_g || !raw_beta || !out) return invalid("mixed_qkv, raw_g, raw_beta and out must be non-NULL");
    if (2 * Hk * K + Hv * V > INT32_MAX)   // columns are counted in 32 bits
        return set_error(KDA_ERR_UNSUPPORTED, "2*Hk*K + Hv*V must be below 2^31 (got %lld)", (long long)(2 * Hk * K + Hv * V));
    if (ld_qkv < 2 * Hk * K + Hv * V)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "ld_qkv (%lld) < 2*Hk*K + Hv*V (%lld)", (long long)ld_qkv, (long long)(2 * Hk * K + Hv * V));
    if (ld_g < Hv || ld_beta < Hv) return invalid("ld_g and ld_beta must be >= Hv");
    if (ld_out < Hv * V) return set_error(KDA_ERR_INVALID_ARGUMENT, "ld_out (%lld) < Hv*V (%lld)", (long long)ld_out, (long long)(Hv * V));
    if (!aligned(out, 8) || ld_out % 4 != 0) return invalid("out must be 8-byte aligned with ld_out a multiple of 4");
    if (!aligned(mixed_qkv, 2) || !aligned(raw_g, 2) || !aligned(raw_beta, 2) || !aligned(hd->A_log, 4) || !aligned(hd->dt_bias, 4) ||
        !aligned(err_flags, 4))
        return invalid("a pointer is not aligned to its element type");
    if (!st) return invalid("state is NULL");
    if (!st->pool || !st->indices) return invalid("state->pool and state->indices must be non-NULL");
    if (st->num_slots < 1) return set_error(KDA_ERR_INVALID_ARGUMENT, "num_slots must be >= 1 (got %lld)", (long long)st->num_slots);
    if (st->slot_stride < Hv * K * V)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "slot_stride (%lld) < Hv*K*V (%lld)", (long long)st->slot_stride, (long long)(Hv * K * V));
    if (st->slot_stride % 4 != 0 || !aligned(st->pool, 16)) return invalid("the pool must be 16-byte aligned and slot_stride a multiple of 4");
    if (st->index_stride < 1) return set_error(KDA_ERR_INVALID_ARGUMENT, "index_stride must be >= 1 (got %lld)", (long long)st->index_stride);
    if (!aligned(st->indices, 4)) return invalid("indices must be 4-byte aligned");
    if (st->null_slot < -1 || st->null_slot >= st->num_slots)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "null_slot must be -1 or in [0, num_slots) (got %d)", st->null_slot);
    if (entries < 0) return invalid("the number of sequences must be >= 0");
    if (entries > INT32_MAX / (4 * Hv))   // one launch has at most four CTAs for an entry and head
        return set_error(KDA_ERR_UNSUPPORTED, "%lld entries x %d heads exceed one launch: split the call", (long long)entries, hd->Hv);
    *p = {mixed_qkv, ld_qkv, raw_g, ld_g, raw_beta, ld_beta, hd->A_log, hd->dt_bias, hd->scale, hd->l2_eps, st->pool, st->num_slots,
          st->slot_stride, st->indices, st->index_stride, st->null_slot, out, ld_out, err_flags, hd->Hk, hd->Hv};
    return KDA_OK;
}

// What a prefill's launches count in 32 bits: rows (a chunk past the last one too), and chunks times heads.
int check_size(int64_t rows, int64_t seqs, int64_t Hv)
{
    if (rows < 0) return invalid("num_rows must be >= 0");
    if (rows > INT32_MAX - 64) return set_error(KDA_ERR_UNSUPPORTED, "num_rows must be below 2^31 - 64 (got %lld)", (long long)rows);
    if (rows / 64 + seqs > INT32_MAX / Hv)
        return set_error(KDA_ERR_UNSUPPORTED, "%lld rows x %lld heads exceed one launch: split the call", (long long)rows, (long long)Hv);
    return KDA_OK;
}

int done(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? set_error(KDA_OK, "%s", "") : set_error(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int kda_gdn_decode(const uint16_t *mixed_qkv, int64_t ld_qkv, const uint16_t *raw_g, int64_t ld_g,
                   const uint16_t *raw_beta, int64_t ld_beta, int64_t num_seqs, const kda_gdn_heads *heads,
                   const kda_state *state, uint16_t *out, int64_t ld_out, uint32_t *err_flags, void *stream)
{
    kda::GdnParams p;
    const int s = check(mixed_qkv, ld_qkv, raw_g, ld_g, raw_beta, ld_beta, num_seqs, heads, state, out, ld_out, err_flags, &p);
    if (s) return s;
    if (num_seqs == 0) return set_error(KDA_OK, "%s", "");
    return done(kda::launch_gdn_decode(p, heads->K, heads->V, num_seqs, static_cast<cudaStream_t>(stream)), "kda_gdn_decode launch");
}

int kda_gdn_spec_verify(const uint16_t *mixed_qkv, int64_t ld_qkv, const uint16_t *raw_g, int64_t ld_g,
                        const uint16_t *raw_beta, int64_t ld_beta, int64_t num_reqs, int32_t tokens_per_req,
                        const kda_gdn_heads *heads, const kda_state *state, uint16_t *out, int64_t ld_out,
                        uint32_t *err_flags, void *stream)
{
    kda::GdnParams p;
    const int s = check(mixed_qkv, ld_qkv, raw_g, ld_g, raw_beta, ld_beta, num_reqs, heads, state, out, ld_out, err_flags, &p);
    if (s) return s;
    if (tokens_per_req < 1 || tokens_per_req > 64)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "tokens_per_req must be in 1..64 (got %d)", tokens_per_req);
    if (num_reqs == 0) return set_error(KDA_OK, "%s", "");
    return done(kda::launch_gdn_rows(p, heads->K, heads->V, tokens_per_req, nullptr, 0, num_reqs, static_cast<cudaStream_t>(stream)),
                "kda_gdn_spec_verify launch");
}

size_t kda_gdn_chunk_prefill_workspace_bytes(int64_t num_rows, int64_t num_seqs, const kda_gdn_heads *heads)
{
    if (!heads) return invalid("heads is NULL"), 0;
    if (heads->Hk < 1 || heads->Hv < 1 || heads->Hv % heads->Hk != 0 || !supported_dim(heads->K) || !supported_dim(heads->V))
        return invalid("Hv must be a multiple of Hk, K and V each 32, 64 or 128"), 0;
    if (num_seqs < 0) return invalid("num_seqs must be >= 0"), 0;
    if (check_size(num_rows, num_seqs, heads->Hv)) return 0;
    set_error(KDA_OK, "%s", "");
    return kda::gdn_prefill_workspace(num_rows, num_seqs, heads->Hv, heads->K, heads->V);
}

int kda_gdn_chunk_prefill(const uint16_t *mixed_qkv, int64_t ld_qkv, const uint16_t *raw_g, int64_t ld_g,
                          const uint16_t *raw_beta, int64_t ld_beta, const int32_t *cu_seqlens, int64_t num_seqs,
                          int64_t num_rows, const kda_gdn_heads *heads, const kda_state *state, void *workspace,
                          size_t workspace_bytes, uint16_t *out, int64_t ld_out, uint32_t *err_flags, void *stream)
{
    kda::GdnParams p;
    const int s = check(mixed_qkv, ld_qkv, raw_g, ld_g, raw_beta, ld_beta, num_seqs, heads, state, out, ld_out, err_flags, &p);
    if (s) return s;
    if (!cu_seqlens || !aligned(cu_seqlens, 4)) return invalid("cu_seqlens must be non-NULL and 4-byte aligned");
    const int r = check_size(num_rows, num_seqs, heads->Hv);
    if (r) return r;
    if (num_seqs == 0 || num_rows == 0) return set_error(KDA_OK, "%s", "");
    const size_t need = kda::gdn_prefill_workspace(num_rows, num_seqs, heads->Hv, heads->K, heads->V);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return set_error(KDA_ERR_WORKSPACE, "kda_gdn_chunk_prefill needs a 256-byte aligned workspace of %zu bytes (got %zu)", need,
                         workspace ? workspace_bytes : static_cast<size_t>(0));
    return done(kda::launch_gdn_prefill(p, heads->K, heads->V, cu_seqlens, num_rows, num_seqs, workspace, static_cast<cudaStream_t>(stream)),
                "kda_gdn_chunk_prefill launch");
}

}  // extern "C"
