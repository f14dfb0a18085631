// gc_rows_internal.h -- the launchers of the row operators (experts.cu,
// embedding.cu, sample.cu) that api_rows.cu dispatches to.  Arguments were
// validated there; strides and widths in elements, `wide`: int64 ids.
#pragma once

#include "gc_internal.h"

namespace gch {

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

}  // namespace gch
