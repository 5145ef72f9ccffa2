// Internal launchers of the operators around the recurrence (batch maps, norm with an 8-bit
// output, 8-bit matrix product), shared by their entry points.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct NormQuantParams {
    const void *x;      int64_t ld_x;
    const void *res;    int64_t ld_res;
    const float *w;     float eps;
    void *res_out;      int64_t ld_ro;
    void *y;            int64_t ld_y;
    uint8_t *q;         int64_t ld_q;
    float *s;           int64_t s_row, s_group;
    int64_t N;          int D;
};
constexpr int kNormMaxCols = 32768;
cudaError_t launch_norm_quant(const NormQuantParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_norm_quant_bf16(const NormQuantParams &p, cudaStream_t stream);
cudaError_t launch_norm_quant_fp16(const NormQuantParams &p, cudaStream_t stream);
cudaError_t launch_norm_quant_fp32(const NormQuantParams &p, cudaStream_t stream);

struct Fp8Params {
    const uint8_t *a;   int64_t ld_a;
    const float *sa;    int64_t sa_row, sa_group;
    const uint8_t *w;   int64_t ld_w;
    const float *sw;    int64_t sw_row, sw_group;
    int M, N, K;
    void *out;          int64_t ld_out;   int out_dtype;
    uint32_t *err;
    int stalled;                         // self-test: the CTA of each cluster whose scales never come (-1: none)
};
cudaError_t launch_fp8_matmul(const Fp8Params &p, cudaStream_t stream);
// Rows of A per tile (0: the general kernel), CTAs that split the inner axis, rows of W per tile.
cudaError_t plan_fp8_matmul(const Fp8Params &p, int32_t (&plan)[3]);

struct BatchMapsParams {
    const int32_t *qlen, *clen;
    const int32_t *slots;      int64_t slot_stride;
    int R;
    int32_t *table;            int64_t table_stride;  int64_t width;
    const int32_t *free_pages; int64_t num_free;      const int32_t *free_count;
    int64_t num_pages;         int page;              int64_t num_tokens;
    int32_t *order, *cu, *state_indices, *num_decodes, *positions;
    int64_t *slot_map;
    int32_t *free_left;
    uint32_t *err;
};
cudaError_t launch_batch_maps(const BatchMapsParams &p, cudaStream_t stream);

}  // namespace kda
