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

// Whether the last of n entries `stride` apart is at less than 2^60.
bool valid_extent(size_t n, size_t stride) { return n <= 1 || stride < (size_t(1) << 60) / n; }

// The rows of a cache: offsets that fit, and for an output no row on another.
bool valid_cache(const gc_cache_rows &c, size_t batch, size_t heads, size_t rows, bool write)
{
    if (c.width < 1 || c.width > GC_MAX_ROW_WIDTH || c.row_stride >= (size_t(1) << 31) ||
        c.head_stride >= (size_t(1) << 48) || c.batch_stride >= (size_t(1) << 48) ||
        !valid_extent(batch, c.batch_stride) || !valid_extent(heads, c.head_stride))
        return false;
    if (!write || batch == 0 || heads == 0 || rows == 0) return true;
    struct {
        size_t n, stride;
    } d[3] = {{rows, c.row_stride}, {heads, c.head_stride}, {batch, c.batch_stride}};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (d[j].stride > d[j + 1].stride) {
                const auto t = d[j];
                d[j] = d[j + 1], d[j + 1] = t;
            }
    size_t reach = c.width;  // elements from a part's first to past its last
    for (const auto &x : d) {
        if (x.n <= 1) continue;
        if (x.stride < reach) return false;
        reach += (x.n - 1) * x.stride;
    }
    return true;
}

Span cache_span(const gc_cache_rows &c, size_t batch, size_t heads, size_t rows, gc_row_dtype dt, bool write)
{
    if (c.d_rows == nullptr || batch == 0 || heads == 0 || rows == 0) return Span{nullptr, 0, row_elem(dt), write};
    const size_t last = (batch - 1) * c.batch_stride + (heads - 1) * c.head_stride + (rows - 1) * c.row_stride + c.width;
    return Span{c.d_rows, last * row_elem(dt), row_elem(dt), write};
}

// CTAs of one launch.
bool valid_grid(size_t a, size_t b) { return b == 0 || a <= GC_MAX_ELEMENTS / b; }

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

size_t gc_expert_route_workspace_bytes(size_t tokens, uint32_t experts)
{
    if (tokens > GC_MAX_ELEMENTS || experts < 1 || experts > GC_MAX_EXPERTS) return 0;
    return expert_route_workspace_bytes(tokens, experts);
}

gc_status gc_expert_route(const void *d_logits, size_t logits_stride, size_t tokens, uint32_t experts,
                          gc_row_dtype dtype, size_t topk, int normalize, const uint8_t *d_mask, int32_t *d_ids,
                          float *d_weights, int32_t *d_counts, float *d_load, float *d_loss, void *d_ws,
                          size_t ws_bytes, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || !valid_routing(tokens, topk) || experts < 1 || experts > GC_MAX_EXPERTS ||
        topk > experts || !valid_rows(tokens, logits_stride, experts))
        return GC_ERR_INVALID_VALUE;
    if ((tokens > 0 && (d_logits == nullptr || d_ids == nullptr || d_weights == nullptr)) ||
        (d_counts == nullptr && (d_load || d_loss)) || d_ws == nullptr)
        return GC_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return GC_ERR_MISALIGNED;
    if (ws_bytes < (d_counts ? expert_route_workspace_bytes(tokens, experts) : 256)) return GC_ERR_WORKSPACE_TOO_SMALL;
    const gc_status st = check_spans({row_span(d_logits, tokens, logits_stride, experts, dtype, false),
                                      flat(d_mask, tokens, 1, false), flat(d_ids, tokens * topk, 4, true),
                                      flat(d_weights, tokens * topk, 4, true),
                                      flat(d_counts, size_t(experts) + 1, 4, true), flat(d_load, experts, 4, true),
                                      flat(d_loss, 1, 4, true), Span{d_ws, ws_bytes, 256, true}});
    if (st != GC_OK || (tokens == 0 && d_counts == nullptr)) return st;
    return from_cuda(launch_expert_route(d_logits, logits_stride, uint32_t(tokens), experts, dtype, uint32_t(topk),
                                         normalize != 0, d_mask, d_ids, d_weights, d_counts, d_load, d_loss,
                                         static_cast<uint8_t *>(d_ws), stream));
}

gc_status gc_expert_route_grad(const void *d_logits, size_t logits_stride, size_t tokens, uint32_t experts,
                               gc_row_dtype dtype, size_t topk, int normalize, const int32_t *d_ids,
                               const int32_t *d_counts, const float *d_dweights, const float *d_dloss, void *d_dx,
                               size_t dx_stride, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || !valid_routing(tokens, topk) || experts < 1 || experts > GC_MAX_EXPERTS ||
        topk > experts || !valid_rows(tokens, logits_stride, experts) || !valid_rows(tokens, dx_stride, experts))
        return GC_ERR_INVALID_VALUE;
    if ((tokens > 0 && (d_logits == nullptr || d_ids == nullptr || d_dx == nullptr)) ||
        (d_dloss != nullptr && d_counts == nullptr))
        return GC_ERR_INVALID_VALUE;
    const gc_status st = check_spans({row_span(d_logits, tokens, logits_stride, experts, dtype, false),
                                      flat(d_ids, tokens * topk, 4, false),
                                      flat(d_counts, size_t(experts) + 1, 4, false),
                                      flat(d_dweights, tokens * topk, 4, false), flat(d_dloss, 1, 4, false),
                                      row_span(d_dx, tokens, dx_stride, experts, dtype, true)});
    if (st != GC_OK || tokens == 0) return st;
    return from_cuda(launch_expert_route_grad(d_logits, logits_stride, uint32_t(tokens), experts, dtype,
                                              uint32_t(topk), normalize != 0, d_ids, d_counts, d_dweights, d_dloss,
                                              d_dx, dx_stride, stream));
}

size_t gc_sample_verify_workspace_bytes(size_t sequences, size_t drafts, size_t vocab)
{
    if (sequences > GC_MAX_ELEMENTS || drafts > GC_MAX_DRAFTS || vocab < 1 || vocab > GC_MAX_SAMPLE_VOCAB) return 0;
    return sample_verify_workspace_bytes(sequences, drafts, vocab);
}

gc_status gc_sample_verify(const void *d_logits, size_t logits_stride, const void *d_draft_logits, size_t draft_stride,
                           size_t sequences, size_t drafts, size_t vocab, gc_row_dtype dtype, const int32_t *d_drafts,
                           const float *d_accept, const float *d_uniform, size_t uniform_stride,
                           const float *d_temperature, int32_t *d_tokens, int32_t *d_accepted, float *d_logprobs,
                           void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    const size_t need = gc_sample_verify_workspace_bytes(sequences, drafts, vocab);
    const size_t rows = sequences * (drafts + 1), drafted = sequences * drafts;
    if (!valid_row_dtype(dtype) || need == 0 || !valid_rows(rows, logits_stride, vocab) ||
        (d_draft_logits && !valid_rows(drafted, draft_stride, vocab)) ||
        (d_uniform && !valid_rows(sequences, uniform_stride, vocab)))
        return GC_ERR_INVALID_VALUE;
    if ((sequences > 0 && (d_logits == nullptr || d_tokens == nullptr || d_accepted == nullptr)) ||
        (drafted > 0 && (d_drafts == nullptr || (d_uniform && d_accept == nullptr))) || d_ws == nullptr)
        return GC_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return GC_ERR_MISALIGNED;
    if (ws_bytes < need) return GC_ERR_WORKSPACE_TOO_SMALL;
    const gc_status st = check_spans({row_span(d_logits, rows, logits_stride, vocab, dtype, false),
                                      row_span(d_draft_logits, drafted, draft_stride, vocab, dtype, false),
                                      flat(d_drafts, drafted, 4, false), flat(d_accept, drafted, 4, false),
                                      row_span(d_uniform, sequences, uniform_stride, vocab, GC_ROW_F32, false),
                                      flat(d_temperature, sequences, 4, false), flat(d_tokens, rows, 4, true),
                                      flat(d_accepted, sequences, 4, true), flat(d_logprobs, rows, 4, true),
                                      Span{d_ws, ws_bytes, 256, true}});
    if (st != GC_OK || sequences == 0) return st;
    return from_cuda(launch_sample_verify(d_logits, logits_stride, drafts ? d_draft_logits : nullptr, draft_stride,
                                          uint32_t(sequences), uint32_t(drafts), uint32_t(vocab), dtype, d_drafts,
                                          d_accept, d_uniform, uniform_stride, d_temperature, d_tokens, d_accepted,
                                          d_logprobs, static_cast<uint8_t *>(d_ws), stream));
}

gc_status gc_cache_score(const void *d_weights, size_t batch_stride, size_t head_stride, size_t query_stride,
                         gc_row_dtype dtype, size_t batch, size_t heads, size_t group, size_t queries, size_t length,
                         const float *d_scores, size_t scores_stride, float decay, const int32_t *d_lengths,
                         const int32_t *d_counted, float *d_out, size_t out_stride, cudaStream_t stream)
{
    if (!valid_row_dtype(dtype) || batch > GC_MAX_ELEMENTS || heads > GC_MAX_ELEMENTS || group < 1 ||
        group > GC_MAX_ELEMENTS || queries > GC_MAX_ELEMENTS || length > GC_MAX_ROW_WIDTH ||
        !valid_grid(batch, heads) || !valid_grid(heads, group) || !valid_grid(group, queries) ||
        !valid_grid(batch * heads, length / 32 + 1) || !valid_extent(batch, batch_stride) ||
        !valid_extent(heads * group, head_stride) || !valid_extent(queries, query_stride))
        return GC_ERR_INVALID_VALUE;
    const size_t rows = batch * heads;
    if (rows == 0 || length == 0) return GC_OK;
    if ((d_scores && !valid_rows(rows, scores_stride, length)) || !valid_rows(rows, out_stride, length) ||
        d_out == nullptr || (queries > 0 && d_weights == nullptr))
        return GC_ERR_INVALID_VALUE;
    Span weights{nullptr, 0, row_elem(dtype), false};
    if (queries > 0) {
        const size_t last = (batch - 1) * batch_stride + (heads * group - 1) * head_stride +
                            (queries - 1) * query_stride + length;
        weights = Span{d_weights, last * row_elem(dtype), row_elem(dtype), false};
    }
    // the scores may be updated in place
    const bool in_place = d_scores == d_out;
    if (in_place && scores_stride != out_stride) return GC_ERR_INVALID_VALUE;
    const gc_status st = check_spans({weights,
                                      in_place ? Span{} : row_span(d_scores, rows, scores_stride, length, GC_ROW_F32, false),
                                      flat(d_lengths, batch, 4, false), flat(d_counted, batch, 4, false),
                                      row_span(d_out, rows, out_stride, length, GC_ROW_F32, true)});
    if (st != GC_OK) return st;
    return from_cuda(launch_cache_score(d_weights, batch_stride, head_stride, query_stride, dtype, uint32_t(batch),
                                        uint32_t(heads), uint32_t(group), uint32_t(queries), uint32_t(length),
                                        d_scores, scores_stride, decay, d_lengths, d_counted, d_out, out_stride,
                                        stream));
}

size_t gc_cache_evict_workspace_bytes(size_t batch, size_t heads, size_t budget)
{
    // without a head no kernel would write the sequences' new lengths
    if (batch > GC_MAX_ELEMENTS || heads < 1 || heads > GC_MAX_ELEMENTS || !valid_grid(batch, heads) || budget < 1 ||
        budget > GC_MAX_ROW_WIDTH || !valid_grid(batch * heads, budget))
        return 0;
    return cache_evict_workspace_bytes(batch * heads, budget);
}

gc_status gc_cache_evict(const gc_cache_rows *keys, const gc_cache_rows *values, gc_row_dtype dtype,
                         const float *d_scores, size_t scores_stride, const int32_t *d_positions,
                         size_t positions_stride, const int32_t *d_lengths, size_t batch, size_t heads, size_t length,
                         size_t budget, size_t sinks, size_t recent, const gc_cache_rows *kept_keys,
                         const gc_cache_rows *kept_values, float *d_kept_scores, int32_t *d_kept_positions,
                         int32_t *d_kept_lengths, void *d_ws, size_t ws_bytes, cudaStream_t stream)
{
    const size_t need = gc_cache_evict_workspace_bytes(batch, heads, budget);
    if (!valid_row_dtype(dtype) || need == 0 || length > GC_MAX_ROW_WIDTH || sinks > budget || recent > budget - sinks ||
        keys == nullptr || kept_keys == nullptr || (values == nullptr) != (kept_values == nullptr))
        return GC_ERR_INVALID_VALUE;
    const size_t rows = batch * heads, there = rows * length;
    if (!valid_grid(rows, 8) || !valid_cache(*keys, batch, heads, length, false) ||
        !valid_cache(*kept_keys, batch, heads, budget, true) || keys->width != kept_keys->width ||
        (values && (!valid_cache(*values, batch, heads, length, false) ||
                    !valid_cache(*kept_values, batch, heads, budget, true) || values->width != kept_values->width)))
        return GC_ERR_INVALID_VALUE;
    if (length > 0 && (!valid_rows(rows, scores_stride, length) ||
                       (d_positions && !valid_rows(rows, positions_stride, length))))
        return GC_ERR_INVALID_VALUE;
    if ((there > 0 && (keys->d_rows == nullptr || d_scores == nullptr || (values && values->d_rows == nullptr))) ||
        (rows > 0 && (kept_keys->d_rows == nullptr || (values && kept_values->d_rows == nullptr) ||
                      d_kept_scores == nullptr || d_kept_positions == nullptr || d_kept_lengths == nullptr)) ||
        d_ws == nullptr)
        return GC_ERR_INVALID_VALUE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return GC_ERR_MISALIGNED;
    if (ws_bytes < need) return GC_ERR_WORKSPACE_TOO_SMALL;
    const gc_status st = check_spans(
        {cache_span(*keys, batch, heads, length, dtype, false),
         values ? cache_span(*values, batch, heads, length, dtype, false) : Span{},
         length ? row_span(d_scores, rows, scores_stride, length, GC_ROW_F32, false) : Span{},
         length ? row_span(d_positions, rows, positions_stride, length, GC_ROW_F32, false) : Span{},
         flat(d_lengths, batch, 4, false), cache_span(*kept_keys, batch, heads, budget, dtype, true),
         values ? cache_span(*kept_values, batch, heads, budget, dtype, true) : Span{},
         flat(d_kept_scores, rows * budget, 4, true), flat(d_kept_positions, rows * budget, 4, true),
         flat(d_kept_lengths, batch, 4, true), Span{d_ws, ws_bytes, 256, true}});
    if (st != GC_OK || rows == 0) return st;
    return from_cuda(launch_cache_evict(keys, values, dtype, d_scores, scores_stride, d_positions, positions_stride,
                                        d_lengths, uint32_t(batch), uint32_t(heads), uint32_t(length),
                                        uint32_t(budget), uint32_t(sinks), uint32_t(recent), kept_keys, kept_values,
                                        d_kept_scores, d_kept_positions, d_kept_lengths,
                                        static_cast<uint8_t *>(d_ws), stream));
}

}  // extern "C"
