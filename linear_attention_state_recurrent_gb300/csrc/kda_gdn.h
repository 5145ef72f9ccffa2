// Internal parameters and launchers of the gated delta rule with one decay per head, shared by its entry points and kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct GdnParams {
    const uint16_t *qkv;    int64_t ld_qkv;     // rows [q (Hk K) | k (Hk K) | v (Hv V)]
    const uint16_t *rg;     int64_t ld_g;
    const uint16_t *rb;     int64_t ld_beta;
    const float *A_log, *dt_bias;
    float scale, eps;
    float *pool;            int64_t num_slots, slot_stride;
    const int32_t *indices; int64_t index_stride; int null_slot;
    uint16_t *out;          int64_t ld_out;
    uint32_t *err;
    int Hk, Hv;
};

// One row per sequence.
cudaError_t launch_gdn_decode(const GdnParams &p, int K, int V, int64_t num_seqs, cudaStream_t stream);

// T rows per entry (cu NULL), or the rows [cu[e], cu[e + 1]) of `rows` packed ones (cu on the device).
cudaError_t launch_gdn_rows(const GdnParams &p, int K, int V, int T, const int32_t *cu, int64_t rows, int64_t num_entries,
                            cudaStream_t stream);

// The rows [cu[e], cu[e + 1]) of `rows` packed ones per sequence, in chunks. Bytes of workspace, and the launches.
size_t gdn_prefill_workspace(int64_t rows, int64_t num_seqs, int Hv, int K, int V);
cudaError_t launch_gdn_prefill(const GdnParams &p, int K, int V, const int32_t *cu, int64_t rows, int64_t num_seqs, void *workspace,
                               cudaStream_t stream);

}  // namespace kda
