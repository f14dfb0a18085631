// embedding.cu -- embedding lookup with scaling (gc_embedding) and its
// gradient by tokens sorted stably (gc_embedding_grad).
//
// The gradient sorts (token, position) pairs by LSD passes of the stable bin
// partition (gc_binsort.cuh), up to 9 bits each, so that every table row's
// positions are contiguous and ascending; then each table row is the sum of
// its positions' rows.  A frequent token's positions are summed in fixed
// blocks first, so that no CTA walks them alone.  Every sum's order depends
// on the ids alone.
#include "gc_binsort.cuh"
#include "gc_internal.h"
#include "gc_rows.cuh"

namespace {

using namespace gcd;

constexpr int kRowThreads = 256;

dim3 row_block(size_t pieces)
{
    int tx = 32;
    while (tx < kRowThreads && size_t(tx) < pieces) tx <<= 1;
    return dim3(tx, kRowThreads / tx);
}

template <class T, int N>
__global__ void __launch_bounds__(kRowThreads)
embedding_kernel(const T *__restrict__ table, size_t table_stride, uint32_t vocab, uint32_t pieces,
                 const void *__restrict__ ids, bool wide, uint32_t n, float scale, T *__restrict__ out,
                 size_t out_stride)
{
    const uint32_t i = blockIdx.x * blockDim.y + threadIdx.y;
    if (i >= n) return;
    const uint32_t id = load_id(ids, wide, i, vocab);
    const T *src = table + size_t(id) * table_stride;
    T *dst = out + size_t(i) * out_stride;
    for (uint32_t c = threadIdx.x; c < pieces; c += blockDim.x) {
        Piece<T, N> v = zero_piece<T, N>();
        if (id < vocab) {
            v = load_piece<T, N>(src + size_t(c) * N);
#pragma unroll
            for (int k = 0; k < N; ++k) v.v[k] = row_from_float<T>(scale * row_to_float(v.v[k]));
        }
        store_piece<T, N>(dst + size_t(c) * N, v);
    }
}

// A pass's items: (key, position) pairs, or in the first pass the ids
// themselves; an id outside the vocabulary is the key `vocab`, which sorts
// last.
struct TokenPass {
    const void *ids;        // first pass
    const uint2 *in;        // later passes
    bool first, wide;
    uint32_t vocab, shift, mask;
    __device__ __forceinline__ uint2 item(uint32_t i) const
    {
        return first ? make_uint2(load_id(ids, wide, i, vocab), i) : in[i];
    }
    __device__ __forceinline__ uint32_t bin(uint32_t i) const { return (item(i).x >> shift) & mask; }
};

struct TokenSink {
    TokenPass src;
    uint2 *out;
    __device__ __forceinline__ void start(uint32_t, uint32_t, uint32_t) const {}
    __device__ __forceinline__ void end(uint32_t) const {}
    __device__ __forceinline__ void place(uint32_t i, uint32_t at) const { out[at] = src.item(i); }
    __device__ __forceinline__ void drop(uint32_t) const {}
};

// [start, end) of every token that occurs, in bounds (zeroed before).
__global__ void __launch_bounds__(256)
token_bounds_kernel(const uint2 *__restrict__ sorted, uint32_t n, uint32_t vocab, uint2 *__restrict__ bounds)
{
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;
    const uint32_t key = sorted[i].x;
    if (key >= vocab) return;
    if (i == 0 || sorted[i - 1].x != key) bounds[key].x = i;
    if (i + 1 == n || sorted[i + 1].x != key) bounds[key].y = i + 1;
}

// Sums of the blocks of `block` sorted positions that hold one token only.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads)
token_blocks_kernel(const uint2 *__restrict__ sorted, uint32_t vocab, uint32_t block, const T *__restrict__ g,
                    size_t g_stride, uint32_t width, float *__restrict__ partial)
{
    const uint32_t first = blockIdx.x * block;
    const uint32_t key = sorted[first].x;
    if (key >= vocab || sorted[first + block - 1].x != key) return;
    const uint32_t c = (blockIdx.y * kRowThreads + threadIdx.x) * N;
    if (c >= width) return;
    float acc[N] = {};
    for (uint32_t i = first; i < first + block; ++i) {
        const Piece<T, N> v = load_piece<T, N>(g + size_t(sorted[i].y) * g_stride + c);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += row_to_float(v.v[k]);
    }
    for (int k = 0; k < N; ++k) partial[size_t(blockIdx.x) * width + c + k] = acc[k];
}

// dtable[v] (+)= scale * (sum of v's rows).
template <class T, class O, int N>
__global__ void __launch_bounds__(kRowThreads)
token_rows_kernel(const uint2 *__restrict__ sorted, const uint2 *__restrict__ bounds, uint32_t vocab,
                  uint32_t block, const T *__restrict__ g, size_t g_stride, uint32_t width,
                  const float *__restrict__ partial, float scale, O *__restrict__ out, size_t out_stride,
                  bool accumulate)
{
    const uint32_t v = blockIdx.x * blockDim.y + threadIdx.y;
    if (v >= vocab) return;
    const uint2 range = bounds[v];
    if (accumulate && range.x == range.y) return;
    for (uint32_t c = threadIdx.x * N; c < width; c += blockDim.x * N) {
        float acc[N] = {};
        for (uint32_t i = range.x; i < range.y;) {
            if (i % block == 0 && i + block <= range.y) {
                const float *p = partial + size_t(i / block) * width + c;
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += p[k];
                i += block;
            } else {
                const Piece<T, N> x = load_piece<T, N>(g + size_t(sorted[i].y) * g_stride + c);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += row_to_float(x.v[k]);
                ++i;
            }
        }
        O *dst = out + size_t(v) * out_stride + c;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float r = scale * acc[k];
            if (accumulate) r += row_to_float(dst[k]);
            dst[k] = row_from_float<O>(r);
        }
    }
}

// Sorted positions per block: about sqrt(n), so that the longest token's sum
// is about sqrt(n) steps in both kernels.
uint32_t token_block(size_t n)
{
    uint32_t b = 32;
    while (size_t(b) * b < n && b < 4096) b <<= 1;
    return b;
}

int key_bits(size_t vocab)
{
    int bits = 1;
    while ((size_t(vocab) >> bits) != 0) ++bits;
    return bits;
}

struct GradLayout {
    size_t items_a, items_b, table, bounds, partial, total;
};

GradLayout grad_layout(size_t n, size_t vocab, size_t width)
{
    GradLayout l{};
    const size_t items = gch::align_up(8 * n, 256);
    l.items_a = 0;
    l.items_b = items;
    l.table = 2 * items;
    l.bounds = l.table + gch::align_up(size_t(bin_chunks(n)) * 512 * 4, 256);
    l.partial = l.bounds + gch::align_up(8 * vocab, 256);
    l.total = l.partial + gch::align_up(n / token_block(n) * width * 4, 256) + 256;
    return l;
}

template <class T, class O, int N>
cudaError_t run_grad_rows(const uint2 *sorted, const uint2 *bounds, uint32_t n, uint32_t vocab, const void *g,
                          size_t g_stride, size_t width, float *partial, float scale, void *out,
                          size_t out_stride, bool accumulate, cudaStream_t s)
{
    const uint32_t block = token_block(n);
    const uint32_t pieces = uint32_t(width / N);
    if (n / block > 0)
        token_blocks_kernel<T, N><<<dim3(n / block, uint32_t(gch::ceil_div(pieces, kRowThreads))), kRowThreads, 0, s>>>(
            sorted, vocab, block, static_cast<const T *>(g), g_stride, uint32_t(width), partial);
    const dim3 threads = row_block(pieces);
    token_rows_kernel<T, O, N><<<uint32_t(gch::ceil_div(vocab, threads.y)), threads, 0, s>>>(
        sorted, bounds, vocab, block, static_cast<const T *>(g), g_stride, uint32_t(width), partial, scale,
        static_cast<O *>(out), out_stride, accumulate);
    return cudaGetLastError();
}

#define GC_BY_PIECE(T, n, CALL)                                     \
    switch (n) {                                                    \
    case 1: CALL(T, 1); break;                                      \
    case 2: CALL(T, 2); break;                                      \
    case 4: CALL(T, 4); break;                                      \
    default: CALL(T, (16 / int(sizeof(T)))); break;                 \
    }

}  // namespace

namespace gch {

size_t embedding_grad_workspace_bytes(size_t n, size_t vocab, size_t width) { return grad_layout(n, vocab, width).total; }

cudaError_t launch_embedding(const void *table, size_t table_stride, uint32_t vocab, size_t width, gc_row_dtype dt,
                             const void *ids, bool wide, uint32_t n, float scale, void *out, size_t out_stride,
                             cudaStream_t s)
{
    const int elem = dt == GC_ROW_F32 ? 4 : 2;
    const int m = piece_elems(uint64_t(uintptr_t(table)) | uintptr_t(out) | elem * (table_stride | out_stride | width),
                              elem);
#define GC_EMBED_CALL(T, N)                                                                                      \
    {                                                                                                            \
        const uint32_t pieces = uint32_t(width / (N));                                                           \
        const dim3 block = row_block(pieces);                                                                    \
        embedding_kernel<T, N><<<uint32_t(ceil_div(n, block.y)), block, 0, s>>>(                                 \
            static_cast<const T *>(table), table_stride, vocab, pieces, ids, wide, n, scale, static_cast<T *>(out), \
            out_stride);                                                                                         \
    }
    if (dt == GC_ROW_F32) { GC_BY_PIECE(float, m, GC_EMBED_CALL) }
    else if (dt == GC_ROW_BF16) { GC_BY_PIECE(__nv_bfloat16, m, GC_EMBED_CALL) }
    else { GC_BY_PIECE(__half, m, GC_EMBED_CALL) }
    return cudaGetLastError();
}

cudaError_t launch_embedding_grad(const void *g, size_t g_stride, gc_row_dtype gdt, const void *ids, bool wide,
                                  uint32_t n, uint32_t vocab, size_t width, float scale, void *out,
                                  size_t out_stride, gc_row_dtype odt, bool accumulate, uint8_t *ws, cudaStream_t s)
{
    const GradLayout l = grad_layout(n, vocab, width);
    uint2 *items[2] = {reinterpret_cast<uint2 *>(ws + l.items_a), reinterpret_cast<uint2 *>(ws + l.items_b)};
    uint32_t *table = reinterpret_cast<uint32_t *>(ws + l.table);
    uint2 *bounds = reinterpret_cast<uint2 *>(ws + l.bounds);
    float *partial = reinterpret_cast<float *>(ws + l.partial);
    cudaError_t e = cudaMemsetAsync(bounds, 0, size_t(vocab) * 8, s);
    if (e != cudaSuccess) return e;
    int at = 0;
    if (n > 0) {
        const int bits = key_bits(vocab), passes = int(ceil_div(bits, 9)), digit = int(ceil_div(bits, passes));
        for (int p = 0; p < passes; ++p) {
            const TokenPass src{ids, items[at], p == 0, wide, vocab, uint32_t(p * digit), (1u << digit) - 1u};
            const TokenSink sink{src, items[at ^ 1]};
            if ((e = gcd::launch_bin_count(src, n, 1u << digit, table, s)) != cudaSuccess) return e;
            if ((e = gcd::launch_bin_place(src, sink, n, 1u << digit, 1u, table, s)) != cudaSuccess) return e;
            at ^= 1;
        }
        token_bounds_kernel<<<uint32_t(ceil_div(n, 256)), 256, 0, s>>>(items[at], n, vocab, bounds);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const int elem = gdt == GC_ROW_F32 ? 4 : 2;
    const int m = piece_elems(uint64_t(uintptr_t(g)) | elem * (g_stride | width), elem);
#define GC_GRAD_ARGS items[at], bounds, n, vocab, g, g_stride, width, partial, scale, out, out_stride, accumulate, s
#define GC_GRAD_WIDE(T, N) e = run_grad_rows<T, float, N>(GC_GRAD_ARGS)
#define GC_GRAD_SAME(T, N) e = run_grad_rows<T, T, N>(GC_GRAD_ARGS)
    if (gdt == GC_ROW_F32) { GC_BY_PIECE(float, m, GC_GRAD_WIDE) }
    else if (gdt == GC_ROW_BF16 && odt == GC_ROW_F32) { GC_BY_PIECE(__nv_bfloat16, m, GC_GRAD_WIDE) }
    else if (gdt == GC_ROW_BF16) { GC_BY_PIECE(__nv_bfloat16, m, GC_GRAD_SAME) }
    else if (odt == GC_ROW_F32) { GC_BY_PIECE(__half, m, GC_GRAD_WIDE) }
    else { GC_BY_PIECE(__half, m, GC_GRAD_SAME) }
    return e;
}

}  // namespace gch
