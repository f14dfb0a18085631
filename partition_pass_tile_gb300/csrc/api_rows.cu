// api_rows.cu -- the C ABI of the row operators (include/gc.h): argument
// checks on the host and dispatch to the launchers.  As in api.cu, nothing
// touches the GPU before every argument has been checked.
#include <initializer_list>

#include "../../include/gc.h"
#include "../../include/gc_testing.h"
#include "gc_rows_internal.h"

namespace {

using namespace gch;

gc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GC_OK : GC_ERR_CUDA; }

bool valid_row_dtype(int dt) { return dt == GC_ROW_F32 || dt == GC_ROW_BF16 || dt == GC_ROW_F16; }
bool valid_id_type(int t) { return t == GC_ID_I32 || t == GC_ID_I64; }
size_t row_elem(gc_row_dtype dt) { return dt == GC_ROW_F32 ? 4 : 2; }

// A byte range that a call reads or writes; empty without a pointer.
struct Span {
    const void *p;
    size_t bytes, align;
    bool write;
};

Span flat(const void *p, size_t n, size_t elem, bool write) { return Span{p, p ? n * elem : 0, elem, write}; }

Span row_span(const void *p, size_t rows, size_t stride, size_t width, gc_row_dtype dt, bool write)
{
    return Span{p, p && rows ? ((rows - 1) * stride + width) * row_elem(dt) : 0, row_elem(dt), write};
}

// Alignment of every span, and no written span overlapping another one.
gc_status check_spans(std::initializer_list<Span> spans)
{
    for (const Span &a : spans)
        if (a.bytes && reinterpret_cast<uintptr_t>(a.p) % a.align != 0) return GC_ERR_MISALIGNED;
    for (const Span &a : spans) {
        if (!a.write || a.bytes == 0) continue;
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p);
        for (const Span &b : spans) {
            if (&a == &b || b.bytes == 0) continue;
            const uintptr_t y = reinterpret_cast<uintptr_t>(b.p);
            if (x < y + b.bytes && y < x + a.bytes) return GC_ERR_INVALID_VALUE;
        }
    }
    return GC_OK;
}

// Rows and strides below 2^31, so no offset of an element overflows 64 bits.
bool valid_rows(size_t rows, size_t stride, size_t width)
{
    return rows <= GC_MAX_ELEMENTS && width >= 1 && width <= GC_MAX_ROW_WIDTH && stride >= width &&
           stride < (size_t(1) << 31);
}

bool valid_routing(size_t tokens, size_t topk)
{
    return topk >= 1 && topk <= GC_MAX_TOPK && tokens <= GC_MAX_ELEMENTS && tokens * topk <= GC_MAX_ELEMENTS;
}

// gc_embedding_grad, with its wait.
gc_status embedding_grad(const void *d_g, size_t g_stride, gc_row_dtype g_dtype, const void *d_ids, gc_id_type id_type,
                         size_t n, size_t vocab, size_t width, float scale, void *d_dtable, size_t dtable_stride,
                         gc_row_dtype out_dtype, int accumulate, void *d_ws, size_t ws_bytes, cudaStream_t stream,
                         const StagedWait &wait = {})
{
    if (!valid_row_dtype(g_dtype) || !valid_id_type(id_type) || !valid_rows(n, g_stride, width) ||
        !valid_rows(vocab, dtable_stride, width) || vocab >= GC_MAX_ELEMENTS)
        return GC_ERR_INVALID_VALUE;
    if (!valid_row_dtype(out_dtype)) return GC_ERR_INVALID_VALUE;
    if (out_dtype != g_dtype && out_dtype != GC_ROW_F32) return GC_ERR_UNSUPPORTED;
    if (d_ws == nullptr || (n > 0 && (d_ids == nullptr || d_g == nullptr)) || (vocab > 0 && d_dtable == nullptr))
        return GC_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return GC_ERR_MISALIGNED;
    if (ws_bytes < embedding_grad_workspace_bytes(n, vocab, width)) return GC_ERR_WORKSPACE_TOO_SMALL;
    const gc_status st = check_spans({row_span(d_g, n, g_stride, width, g_dtype, false),
                                      flat(d_ids, n, id_type == GC_ID_I64 ? 8 : 4, false),
                                      row_span(d_dtable, vocab, dtable_stride, width, out_dtype, true),
                                      Span{d_ws, ws_bytes, 256, true}});
    if (st != GC_OK) return st;
    return from_cuda(launch_embedding_grad(d_g, g_stride, g_dtype, d_ids, id_type == GC_ID_I64, uint32_t(n),
                                           uint32_t(vocab), width, scale, d_dtable, dtable_stride, out_dtype,
                                           accumulate != 0, static_cast<uint8_t *>(d_ws), stream, wait));
}

}  // namespace

extern "C" {

size_t gc_expert_rows(size_t tokens, size_t topk, uint32_t experts, uint32_t align)
{
    if (!valid_routing(tokens, topk) || experts < 1 || experts > GC_MAX_EXPERTS || align < 1 ||
        align > GC_MAX_EXPERT_ALIGN)
        return 0;
    const size_t pairs = tokens * topk;
    const size_t rows = pairs + (pairs < experts ? pairs : experts) * size_t(align - 1);
    return rows <= GC_MAX_ELEMENTS ? rows : 0;
}

size_t gc_expert_workspace_bytes(size_t tokens, size_t topk, uint32_t experts)
{
    if (!valid_routing(tokens, topk) || experts < 1 || experts > GC_MAX_EXPERTS) return 0;
    return expert_workspace_bytes(tokens * topk, experts);
}

gc_status gc_expert_dispatch(const void *d_ids, gc_id_type id_type, size_t tokens, size_t topk,
                             uint32_t experts, uint32_t align, const void *d_x, size_t x_stride,
                             size_t width, gc_row_dtype dtype, void *d_out, size_t out_stride,
                             size_t rows, int32_t *d_offsets, int32_t *d_counts, int32_t *d_slots,
                             int32_t *d_pairs, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!valid_id_type(id_type) || !valid_routing(tokens, topk)) return GC_ERR_INVALID_VALUE;
    const size_t npairs = tokens * topk, need = gc_expert_rows(tokens, topk, experts, align);
    if (experts < 1 || experts > GC_MAX_EXPERTS || align < 1 || align > GC_MAX_EXPERT_ALIGN ||
        (npairs > 0 && need == 0) || rows < need || rows > GC_MAX_ELEMENTS)
        return GC_ERR_INVALID_VALUE;
    const bool move = d_out != nullptr;
    if (move != (d_x != nullptr) && !(move && tokens == 0)) return GC_ERR_INVALID_VALUE;
    if (move && (!valid_row_dtype(dtype) || !valid_rows(tokens, x_stride, width) ||
                 !valid_rows(rows, out_stride, width)))
        return GC_ERR_INVALID_VALUE;
    if ((npairs > 0 && (d_ids == nullptr || d_slots == nullptr)) || d_offsets == nullptr || d_counts == nullptr ||
        (rows > 0 && d_pairs == nullptr) || d_ws == nullptr)
        return GC_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return GC_ERR_MISALIGNED;
    if (ws_bytes < expert_workspace_bytes(npairs, experts)) return GC_ERR_WORKSPACE_TOO_SMALL;
    const gc_status st = check_spans({
        flat(d_ids, npairs, id_type == GC_ID_I64 ? 8 : 4, false),
        move ? row_span(d_x, tokens, x_stride, width, dtype, false) : Span{},
        move ? row_span(d_out, rows, out_stride, width, dtype, true) : Span{},
        flat(d_offsets, size_t(experts) + 1, 4, true), flat(d_counts, experts, 4, true),
        flat(d_slots, npairs, 4, true), flat(d_pairs, rows, 4, true), Span{d_ws, ws_bytes, 256, true}});
    if (st != GC_OK) return st;
    return from_cuda(launch_expert_dispatch(d_ids, id_type == GC_ID_I64, uint32_t(npairs), uint32_t(topk), experts,
                                            align, d_x, x_stride, width, dtype, d_out, out_stride, uint32_t(rows),
                                            d_offsets, d_counts, d_slots, d_pairs, static_cast<uint8_t *>(d_ws),
                                            stream));
}

gc_status gc_expert_combine(const void *d_y, size_t y_stride, size_t rows, const int32_t *d_slots,
                            const float *d_weights, size_t tokens, size_t topk, size_t width,
                            gc_row_dtype dtype, void *d_out, size_t out_stride, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || !valid_routing(tokens, topk) || !valid_rows(rows, y_stride, width) ||
        !valid_rows(tokens, out_stride, width))
        return GC_ERR_INVALID_VALUE;
    if (tokens > 0 && (d_slots == nullptr || d_out == nullptr || (rows > 0 && d_y == nullptr)))
        return GC_ERR_INVALID_VALUE;
    const size_t npairs = tokens * topk;
    const gc_status st = check_spans({row_span(d_y, rows, y_stride, width, dtype, false),
                                      flat(d_slots, npairs, 4, false), flat(d_weights, npairs, 4, false),
                                      row_span(d_out, tokens, out_stride, width, dtype, true)});
    if (st != GC_OK || tokens == 0) return st;
    return from_cuda(launch_expert_combine(d_y, y_stride, uint32_t(rows), d_slots, d_weights, uint32_t(tokens),
                                           uint32_t(topk), width, dtype, d_out, out_stride, stream));
}

gc_status gc_expert_combine_grad(const void *d_g, size_t g_stride, const void *d_y, size_t y_stride, size_t rows,
                                 const int32_t *d_slots, const int32_t *d_pairs, const float *d_weights,
                                 size_t tokens, size_t topk, size_t width, gc_row_dtype dtype, void *d_dy,
                                 size_t dy_stride, float *d_dweights, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || !valid_routing(tokens, topk) || !valid_rows(tokens, g_stride, width) ||
        !valid_rows(rows, dy_stride, width) || (d_dweights && !valid_rows(rows, y_stride, width)))
        return GC_ERR_INVALID_VALUE;
    if ((tokens > 0 && (d_g == nullptr || d_slots == nullptr)) ||
        (rows > 0 && (d_pairs == nullptr || d_dy == nullptr || (d_dweights && tokens > 0 && d_y == nullptr))))
        return GC_ERR_INVALID_VALUE;
    const size_t npairs = tokens * topk;
    const gc_status st = check_spans(
        {row_span(d_g, tokens, g_stride, width, dtype, false),
         d_dweights ? row_span(d_y, rows, y_stride, width, dtype, false) : Span{}, flat(d_slots, npairs, 4, false),
         flat(d_pairs, rows, 4, false), flat(d_weights, npairs, 4, false),
         row_span(d_dy, rows, dy_stride, width, dtype, true), flat(d_dweights, npairs, 4, true)});
    if (st != GC_OK || (npairs == 0 && rows == 0)) return st;
    return from_cuda(launch_expert_combine_grad(d_g, g_stride, d_y, y_stride, uint32_t(rows), d_slots, d_pairs,
                                                d_weights, uint32_t(tokens), uint32_t(topk), width, dtype, d_dy,
                                                dy_stride, d_dweights, stream));
}

gc_status gc_embedding(const void *d_table, size_t table_stride, size_t vocab, size_t width, gc_row_dtype dtype,
                       const void *d_ids, gc_id_type id_type, size_t n, float scale, void *d_out,
                       size_t out_stride, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || !valid_id_type(id_type) || !valid_rows(vocab, table_stride, width) ||
        !valid_rows(n, out_stride, width))
        return GC_ERR_INVALID_VALUE;
    if (n > 0 && (d_ids == nullptr || d_out == nullptr || (vocab > 0 && d_table == nullptr)))
        return GC_ERR_INVALID_VALUE;
    const gc_status st = check_spans({row_span(d_table, vocab, table_stride, width, dtype, false),
                                      flat(d_ids, n, id_type == GC_ID_I64 ? 8 : 4, false),
                                      row_span(d_out, n, out_stride, width, dtype, true)});
    if (st != GC_OK || n == 0) return st;
    return from_cuda(launch_embedding(d_table, table_stride, uint32_t(vocab), width, dtype, d_ids,
                                      id_type == GC_ID_I64, uint32_t(n), scale, d_out, out_stride, stream));
}

size_t gc_embedding_grad_workspace_bytes(size_t n, size_t vocab, size_t width)
{
    if (n > GC_MAX_ELEMENTS || vocab >= GC_MAX_ELEMENTS || width < 1 || width > GC_MAX_ROW_WIDTH) return 0;
    return embedding_grad_workspace_bytes(n, vocab, width);
}

gc_status gc_embedding_grad(const void *d_g, size_t g_stride, gc_row_dtype g_dtype, const void *d_ids,
                            gc_id_type id_type, size_t n, size_t vocab, size_t width, float scale, void *d_dtable,
                            size_t dtable_stride, gc_row_dtype out_dtype, int accumulate, void *d_ws,
                            size_t ws_bytes, cudaStream_t stream)
{
    return embedding_grad(d_g, g_stride, g_dtype, d_ids, id_type, n, vocab, width, scale, d_dtable, dtable_stride,
                          out_dtype, accumulate, d_ws, ws_bytes, stream);
}

gc_status gc_testing_embedding_grad_stalled(const void *d_g, size_t g_stride, gc_row_dtype g_dtype, const void *d_ids,
                                            gc_id_type id_type, size_t n, size_t vocab, size_t width, float scale,
                                            void *d_dtable, size_t dtable_stride, gc_row_dtype out_dtype,
                                            int accumulate, void *d_ws, size_t ws_bytes, uint64_t timeout_ns,
                                            cudaStream_t stream)
{
    StagedWait wait;
    wait.timeout_ns = timeout_ns;
    wait.missing = 16;
    return embedding_grad(d_g, g_stride, g_dtype, d_ids, id_type, n, vocab, width, scale, d_dtable, dtable_stride,
                          out_dtype, accumulate, d_ws, ws_bytes, stream, wait);
}

gc_status gc_sample(const void *d_logits, size_t logits_stride, size_t rows, size_t vocab, gc_row_dtype dtype,
                    const float *d_uniform, size_t uniform_stride, const float *d_temperature,
                    const int32_t *d_top_k, const float *d_top_p, const float *d_min_p, int32_t *d_tokens,
                    float *d_logprobs, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || rows > GC_MAX_ELEMENTS || vocab < 1 || vocab > GC_MAX_SAMPLE_VOCAB ||
        !valid_rows(rows, logits_stride, vocab) || (d_uniform && !valid_rows(rows, uniform_stride, vocab)))
        return GC_ERR_INVALID_VALUE;
    if (rows > 0 && (d_logits == nullptr || d_tokens == nullptr)) return GC_ERR_INVALID_VALUE;
    const gc_status st = check_spans({row_span(d_logits, rows, logits_stride, vocab, dtype, false),
                                      row_span(d_uniform, rows, uniform_stride, vocab, GC_ROW_F32, false),
                                      flat(d_temperature, rows, 4, false), flat(d_top_k, rows, 4, false),
                                      flat(d_top_p, rows, 4, false), flat(d_min_p, rows, 4, false),
                                      flat(d_tokens, rows, 4, true), flat(d_logprobs, rows, 4, true)});
    if (st != GC_OK || rows == 0) return st;
    return from_cuda(launch_sample(d_logits, logits_stride, uint32_t(rows), uint32_t(vocab), dtype, d_uniform,
                                   uniform_stride, d_temperature, d_top_k, d_top_p, d_min_p, d_tokens, d_logprobs,
                                   stream));
}

}  // extern "C"
