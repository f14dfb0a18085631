// gc_rows_internal.h -- the launchers of the row operators (experts.cu,
// route.cu, embedding.cu, sample.cu, verify.cu, cache.cu) that api_rows.cu dispatches to.  Arguments were
// validated there; strides and widths in elements, `wide`: int64 ids.
#pragma once

#include "gc_internal.h"

namespace gch {

// SMs that grids, and with them the order of sums, are planned for: sums and
// workspaces do not depend on the device that a call finds.
constexpr size_t kSms = 152;

size_t expert_workspace_bytes(size_t npairs, uint32_t experts);
cudaError_t launch_expert_dispatch(const void *ids, bool wide, uint32_t npairs, uint32_t topk, uint32_t experts,
                                   uint32_t align, const void *x, size_t x_stride, size_t width, gc_row_dtype dt,
                                   void *out, size_t out_stride, uint32_t rows, int32_t *offsets, int32_t *counts,
                                   int32_t *slots, int32_t *pairs, uint8_t *ws, cudaStream_t s);
cudaError_t launch_expert_combine(const void *y, size_t y_stride, uint32_t rows, const int32_t *slots,
                                  const float *weights, uint32_t tokens, uint32_t topk, size_t width,
                                  gc_row_dtype dt, void *out, size_t out_stride, cudaStream_t s);
cudaError_t launch_expert_combine_grad(const void *g, size_t g_stride, const void *y, size_t y_stride, uint32_t rows,
                                       const int32_t *slots, const int32_t *pairs, const float *weights,
                                       uint32_t tokens, uint32_t topk, size_t width, gc_row_dtype dt, void *dy,
                                       size_t dy_stride, float *dweights, cudaStream_t s);
cudaError_t launch_embedding(const void *table, size_t table_stride, uint32_t vocab, size_t width, gc_row_dtype dt,
                             const void *ids, bool wide, uint32_t n, float scale, void *out, size_t out_stride,
                             cudaStream_t s);
// The gradient's wait for its bulk copies; `missing`: bytes waited for that
// nobody copies, which makes it run out.
struct StagedWait {
    uint64_t timeout_ns = LaunchOpts{}.timeout_ns;
    uint32_t missing = 0;
};
size_t embedding_grad_workspace_bytes(size_t n, size_t vocab, size_t width);
cudaError_t launch_embedding_grad(const void *g, size_t g_stride, gc_row_dtype gdt, const void *ids, bool wide,
                                  uint32_t n, uint32_t vocab, size_t width, float scale, void *out,
                                  size_t out_stride, gc_row_dtype odt, bool accumulate, uint8_t *ws, cudaStream_t s,
                                  const StagedWait &wait = {});
cudaError_t launch_sample(const void *logits, size_t logits_stride, uint32_t rows, uint32_t vocab, gc_row_dtype dt,
                          const float *uniform, size_t uniform_stride, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                          float *logprobs, cudaStream_t s);
size_t expert_route_workspace_bytes(size_t tokens, uint32_t experts);
cudaError_t launch_expert_route(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, gc_row_dtype dt,
                                uint32_t topk, bool normalize, const uint8_t *mask, int32_t *ids, float *weights,
                                int32_t *counts, float *load, float *loss, uint8_t *ws, cudaStream_t s);
cudaError_t launch_expert_route_grad(const void *logits, size_t stride, uint32_t tokens, uint32_t experts,
                                     gc_row_dtype dt, uint32_t topk, bool normalize, const int32_t *ids,
                                     const int32_t *counts, const float *dweights, const float *dloss, void *dx,
                                     size_t dx_stride, cudaStream_t s);
size_t sample_verify_workspace_bytes(size_t sequences, size_t drafts, size_t vocab);  // 0: too many rows
cudaError_t launch_sample_verify(const void *logits, size_t logits_stride, const void *draft_logits,
                                 size_t draft_stride, uint32_t sequences, uint32_t drafts, uint32_t vocab,
                                 gc_row_dtype dt, const int32_t *ids, const float *accept, const float *uniform,
                                 size_t uniform_stride, const float *temperature, int32_t *tokens, int32_t *accepted,
                                 float *logprobs, uint8_t *ws, cudaStream_t s);
cudaError_t launch_cache_score(const void *weights, size_t batch_stride, size_t head_stride, size_t query_stride,
                               gc_row_dtype dt, uint32_t batch, uint32_t heads, uint32_t group, uint32_t queries,
                               uint32_t length, const float *scores, size_t scores_stride, float decay,
                               const int32_t *lengths, const int32_t *counted, float *out, size_t out_stride,
                               cudaStream_t s);
size_t cache_evict_workspace_bytes(size_t rows, size_t budget);
cudaError_t launch_cache_evict(const gc_cache_rows *keys, const gc_cache_rows *values, gc_row_dtype dt,
                               const float *scores, size_t scores_stride, const int32_t *positions,
                               size_t positions_stride, const int32_t *lengths, uint32_t batch, uint32_t heads,
                               uint32_t length, uint32_t budget, uint32_t sinks, uint32_t recent,
                               const gc_cache_rows *kept_keys, const gc_cache_rows *kept_values, float *kept_scores,
                               int32_t *kept_positions, int32_t *kept_lengths, uint8_t *ws, cudaStream_t s);

}  // namespace gch
