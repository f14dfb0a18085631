// embedding.cu -- embedding lookup with scaling (gc_embedding) and its
// gradient by tokens sorted stably (gc_embedding_grad).
//
// The gradient sorts (token, position) pairs by LSD passes of the stable bin
// partition (gc_binsort.cuh), up to 9 bits each, so that every table row's
// positions are contiguous and ascending.  Blocks of kBlock sorted positions
// are then summed run by run, whatever tokens they hold, so that a frequent
// token's thousands of rows are spread over the GPU: a run that lies within
// its block is a row of the result, the ends of one that does not are kept
// and joined by a last kernel.  Rows of absent tokens are zeroed beside the
// sums.  Every sum's order depends on the ids alone.
#include "gc_binsort.cuh"
#include "gc_internal.h"
#include "gc_rows.cuh"

namespace {

using namespace gcd;

constexpr int kRowThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kBlock = 32;     // sorted positions per block
#ifndef GC_SUMS_CTAS
#define GC_SUMS_CTAS 4
#endif
constexpr int kLookups = 4;         // rows per thread of a lookup
constexpr size_t kZeroBytes = 32768;  // zeroed per CTA, about

// tx threads across a row's pieces, kRowThreads / tx rows.
dim3 row_block(size_t pieces)
{
    int tx = 32;
    while (tx < kRowThreads && size_t(tx) < pieces) tx <<= 1;
    return dim3(tx, kRowThreads / tx);
}

// A thread moves the same piece of kLookups rows, whose ids and then whose
// pieces are loaded together.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads)
embedding_kernel(const T *__restrict__ table, size_t table_stride, uint32_t vocab, uint32_t pieces,
                 const void *__restrict__ ids, bool wide, uint32_t n, float scale, T *__restrict__ out,
                 size_t out_stride)
{
    const uint32_t first = (blockIdx.x * blockDim.y + threadIdx.y) * kLookups;
    uint32_t id[kLookups];
#pragma unroll
    for (int r = 0; r < kLookups; ++r) id[r] = first + r < n ? load_id(ids, wide, first + r, vocab) : vocab;
    for (uint32_t c = threadIdx.x; c < pieces; c += blockDim.x) {
        Piece<T, N> v[kLookups];
#pragma unroll
        for (int r = 0; r < kLookups; ++r) {
            v[r] = zero_piece<T, N>();
            if (id[r] < vocab) v[r] = load_piece<T, N>(table + size_t(id[r]) * table_stride + size_t(c) * N);
        }
#pragma unroll
        for (int r = 0; r < kLookups; ++r) {
            if (id[r] < vocab)  // zeros stay zeros whatever the scale
#pragma unroll
                for (int k = 0; k < N; ++k) v[r].v[k] = row_from_float<T>(scale * row_to_float(v[r].v[k]));
            if (first + r < n) store_piece<T, N>(out + size_t(first + r) * out_stride + size_t(c) * N, v[r]);
        }
    }
}

// A pass's items: (key, position) pairs, or in the first pass the ids
// themselves; an id outside the vocabulary is the key `vocab`, which sorts
// last.  The first pass marks the tokens that occur.
struct TokenPass {
    const void *ids;        // first pass
    const uint2 *in;        // later passes
    uint8_t *seen;          // may be null
    bool first, wide;
    uint32_t vocab, shift, mask;
    __device__ __forceinline__ uint2 item(uint32_t i) const
    {
        return first ? make_uint2(load_id(ids, wide, i, vocab), i) : in[i];
    }
    __device__ __forceinline__ uint32_t bin(uint32_t i) const { return (item(i).x >> shift) & mask; }
    __device__ __forceinline__ void visit(uint32_t i) const
    {
        if (!first || seen == nullptr) return;
        const uint32_t key = load_id(ids, wide, i, vocab);
        if (key < vocab) seen[key] = 1;
    }
};

struct TokenSink {
    TokenPass src;
    uint2 *out;
    __device__ __forceinline__ void start(uint32_t, uint32_t, uint32_t) const {}
    __device__ __forceinline__ void end(uint32_t) const {}
    __device__ __forceinline__ void place(uint32_t i, uint32_t at) const { out[at] = src.item(i); }
    __device__ __forceinline__ void drop(uint32_t) const {}
};

// A short sort, and the clearing of `seen`, by one CTA: the items stay in
// shared memory between the passes.
struct TokenSortSmem {
    BinSmem bins;
    uint2 items[2][kBinSingle];
    uint32_t cnt[kBinWarps << 9];
};

__global__ void __launch_bounds__(kBinThreads)
token_sort_kernel(const void *ids, bool wide, uint32_t n, uint32_t vocab, uint32_t digit, int passes, uint2 *sorted,
                  uint8_t *seen)
{
    extern __shared__ __align__(16) uint8_t token_smem[];
    TokenSortSmem &sm = *reinterpret_cast<TokenSortSmem *>(token_smem);
    if (seen != nullptr)
        for (uint32_t i = threadIdx.x; i < (vocab + 15u) / 16u; i += kBinThreads)  // `seen` has room for whole words
            reinterpret_cast<uint4 *>(seen)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (uint32_t i = threadIdx.x; i < n; i += kBinThreads) sm.items[0][i] = make_uint2(load_id(ids, wide, i, vocab), i);
    __syncthreads();
    if (seen != nullptr)
        for (uint32_t i = threadIdx.x; i < n; i += kBinThreads)
            if (sm.items[0][i].x < vocab) seen[sm.items[0][i].x] = 1;
    for (int p = 0; p < passes; ++p) {
        const TokenPass src{nullptr, sm.items[p & 1], nullptr, false, wide, vocab, uint32_t(p) * digit,
                            (1u << digit) - 1u};
        const TokenSink sink{src, p + 1 < passes ? sm.items[(p & 1) ^ 1] : sorted};
        bin_place_chunk(src, sink, n, n, 1, 0, 1u << digit, 1u, nullptr, sm.cnt, sm.bins);
        __syncthreads();
    }
}

template <class O, int N>
__device__ __forceinline__ void put_sum(O *dst, const float (&sum)[N], float scale, bool accumulate)
{
    Piece<O, N> o;
    if (accumulate) o = load_piece<O, N>(dst);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float r = scale * sum[k];
        o.v[k] = row_from_float<O>(accumulate ? r + row_to_float(o.v[k]) : r);
    }
    store_piece<O, N>(dst, o);
}

struct GradOut {
    void *rows;
    size_t stride;
    float scale;
    bool accumulate;
    const uint8_t *seen;
    uint32_t vocab;
};

// CTAs below `sums`: blocks of kBlock sorted positions, one to a row of
// threads, summed run by run.  edges: two rows per block, the sum of its
// first run where that began before the block, and of its last where that
// began in the block and goes on.  The other CTAs zero rows of absent tokens.
// The rows of the next kAhead positions, and what they are added to, are
// loaded while the ones before are summed.
template <class T, class O, int N, bool ADD>
__global__ void __launch_bounds__(kRowThreads, GC_SUMS_CTAS)
token_sums_kernel(const uint2 *__restrict__ sorted, uint32_t n, const T *__restrict__ g, size_t g_stride,
                  uint32_t width, float *__restrict__ edges, GradOut out, uint32_t sums, uint32_t zero_rows)
{
    O *rows = static_cast<O *>(out.rows);
    const uint32_t columns = blockDim.x * N;
    if (blockIdx.x >= sums) {
        const uint32_t first = (blockIdx.x - sums) * zero_rows, last = min(out.vocab, first + zero_rows);
        for (uint32_t v = first + threadIdx.y; v < last; v += blockDim.y) {
            if (out.seen[v]) continue;
            for (uint32_t c = threadIdx.x * N; c < width; c += columns)
                store_piece<O, N>(rows + size_t(v) * out.stride + c, zero_piece<O, N>());
        }
        return;
    }
    // Keys of the block's positions between those of its neighbours, and the
    // positions; none: the end of the tokens in range.
    __shared__ uint32_t s_key[kRowThreads / 32][kBlock + 2], s_at[kRowThreads / 32][kBlock];
    const uint32_t parts = (width + columns - 1) / columns;  // of a row, neighbours in the grid
    const uint32_t block = blockIdx.x / parts * blockDim.y + threadIdx.y, first = block * kBlock;
    const uint32_t none = out.vocab;
    uint32_t *key = s_key[threadIdx.y], *at = s_at[threadIdx.y];
    for (uint32_t j = threadIdx.x; j < kBlock + 2; j += blockDim.x) {
        const uint32_t i = first + j - 1;  // wraps before the first
        const uint2 item = i < n ? sorted[i] : make_uint2(none, 0u);
        key[j] = item.x;
        if (j >= 1 && j <= kBlock) at[j - 1] = item.y;
    }
    __syncthreads();
    const uint32_t c = (blockIdx.x % parts) * columns + threadIdx.x * N;
    if (key[1] == none || c >= width) return;
    constexpr int kAhead = ADD ? 4 : 8;
    Piece<T, N> x[kAhead];
    Piece<O, N> old[ADD ? kAhead : 1];
    auto load = [&](uint32_t base) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t k = base + j < kBlock ? key[base + j + 1] : none;
            if (k == none) continue;
            x[j] = load_piece<T, N>(g + size_t(at[base + j]) * g_stride + c);
            if (ADD && key[base + j + 2] != k) old[ADD ? j : 0] = load_piece<O, N>(rows + size_t(k) * out.stride + c);
        }
    };
    Piece<float, N> sum{};
    bool began = key[0] != key[1];
    load(0);
    for (uint32_t base = 0; base < kBlock; base += kAhead) {
        Piece<T, N> now[kAhead];
        Piece<O, N> add[ADD ? kAhead : 1];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            now[j] = x[j];
            if (ADD) add[j] = old[j];
        }
        load(base + kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t k = key[base + j + 1];
            if (k == none) return;
#pragma unroll
            for (int e = 0; e < N; ++e) sum.v[e] += row_to_float(now[j].v[e]);
            const bool ends = key[base + j + 2] != k;
            if (ends && began) {
                Piece<O, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float r = out.scale * sum.v[e];
                    o.v[e] = row_from_float<O>(ADD ? r + row_to_float(add[ADD ? j : 0].v[e]) : r);
                }
                store_piece<O, N>(rows + size_t(k) * out.stride + c, o);
            } else if (ends || base + j + 1 == kBlock) {
                store_piece<float, N>(edges + (size_t(block) * 2 + (began ? 1 : 0)) * width + c, sum);
            }
            if (ends) {
                sum = Piece<float, N>{};
                began = true;
            }
        }
    }
}

// Tokens whose run crosses blocks: the block in which it began adds up its
// parts.
template <class O, int N>
__global__ void __launch_bounds__(kRowThreads)
token_join_kernel(const uint2 *__restrict__ sorted, uint32_t n, uint32_t width, const float *__restrict__ edges,
                  GradOut out)
{
    const uint32_t columns = blockDim.x * N, parts = (width + columns - 1) / columns;
    const uint32_t block = blockIdx.x / parts * blockDim.y + threadIdx.y;
    const uint32_t c = (blockIdx.x % parts) * columns + threadIdx.x * N;
    const uint32_t blocks = (n + kBlock - 1) / kBlock;
    if (block + 1 >= blocks) return;  // as does its whole warp
    const uint32_t first = block * kBlock, next = first + kBlock;
    const uint32_t key = sorted[next - 1].x;
    if (key >= out.vocab || sorted[next].x != key || (first > 0 && sorted[first - 1].x == key)) return;
    // The blocks whose first key is it: the run reaches them.
    uint32_t more = 1;
    for (bool on = true; on; ) {
        const uint32_t b = block + more + 1 + (threadIdx.x & 31);
        const uint32_t same = __ballot_sync(kFull, b < blocks && sorted[size_t(min(b, blocks - 1)) * kBlock].x == key);
        more += uint32_t(__ffs(~same) == 0 ? 32 : __ffs(~same) - 1);
        on = same == kFull;
    }
    if (c >= width) return;
    const uint32_t lo = block + more;
    constexpr int kAhead = 8;
    const float *e = edges + (size_t(block) * 2 + 1) * width + c;
    Piece<float, N> sum = load_piece<float, N>(e);
    e += width;
    for (uint32_t b = block + 1; b <= lo; b += kAhead) {
        Piece<float, N> x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            x[j] = Piece<float, N>{};
            if (b + j <= lo) x[j] = load_piece<float, N>(e + size_t(j) * 2 * width);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int k = 0; k < N; ++k) sum.v[k] += x[j].v[k];
        e += size_t(kAhead) * 2 * width;
    }
    put_sum<O, N>(static_cast<O *>(out.rows) + size_t(key) * out.stride + c, sum.v, out.scale, out.accumulate);
}

int key_bits(size_t vocab)
{
    int bits = 1;
    while ((size_t(vocab) >> bits) != 0) ++bits;
    return bits;
}

struct GradLayout {
    size_t items_a, items_b, table, seen, edges, total;
};

GradLayout grad_layout(size_t n, size_t vocab, size_t width)
{
    GradLayout l{};
    const size_t items = gch::align_up(8 * n, 256);
    l.items_a = 0;
    l.items_b = items;
    l.table = 2 * items;
    l.seen = l.table + gch::align_up(bin_table_bytes(n, 512), 256);
    l.edges = l.seen + gch::align_up(vocab, 256);
    l.total = l.edges + gch::align_up(gch::ceil_div(n, size_t(kBlock)) * 2 * width * 4, 256) + 256;
    return l;
}

template <class T, class O, int N>
cudaError_t run_grad_rows(const uint2 *sorted, uint32_t n, const void *g, size_t g_stride, size_t width,
                          float *edges, const GradOut &out, cudaStream_t s)
{
    const dim3 threads = row_block(width / N);
    const uint32_t blocks = uint32_t(gch::ceil_div(n, kBlock));
    const size_t parts = gch::ceil_div(width / N, threads.x);
    const size_t sums = gch::ceil_div(blocks, threads.y) * parts;
    const size_t zero_rows = gch::align_up(gch::ceil_div(kZeroBytes, width * sizeof(O)), threads.y);
    const size_t zeros = out.accumulate ? 0 : gch::ceil_div(out.vocab, zero_rows);
    if (sums + zeros > 0x7fffffffu) return cudaErrorInvalidConfiguration;
    auto kernel = out.accumulate ? token_sums_kernel<T, O, N, true> : token_sums_kernel<T, O, N, false>;
    if (sums + zeros > 0)
        kernel<<<uint32_t(sums + zeros), threads, 0, s>>>(sorted, n, static_cast<const T *>(g), g_stride,
                                                          uint32_t(width), edges, out, uint32_t(sums),
                                                          uint32_t(zero_rows));
    if (blocks > 1)
        token_join_kernel<O, N><<<uint32_t(sums), threads, 0, s>>>(sorted, n, uint32_t(width), edges, out);
    return cudaGetLastError();
}

// Pieces of N elements, N a power of two that both rows allow and that fills
// 16 bytes of the result at most.
#define GC_GRAD_BY_PIECE(T, O, n)                                                   \
    switch (n) {                                                                    \
    case 1: return run_grad_rows<T, O, 1>(sorted, n_, g, g_stride, width, edges, out, s); \
    case 2: return run_grad_rows<T, O, 2>(sorted, n_, g, g_stride, width, edges, out, s); \
    case 4: return run_grad_rows<T, O, 4>(sorted, n_, g, g_stride, width, edges, out, s); \
    default: return run_grad_rows<T, O, 16 / int(sizeof(O))>(sorted, n_, g, g_stride, width, edges, out, s); \
    }

template <class T, class O>
cudaError_t grad_rows(const uint2 *sorted, uint32_t n_, const void *g, size_t g_stride, size_t width, float *edges,
                      const GradOut &out, cudaStream_t s)
{
    const int in = gch::piece_elems(uint64_t(uintptr_t(g)) | sizeof(T) * (g_stride | width), sizeof(T));
    const int to = gch::piece_elems(uint64_t(uintptr_t(out.rows)) | sizeof(O) * (out.stride | width), sizeof(O));
    GC_GRAD_BY_PIECE(T, O, (in < to ? in : to))
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
        embedding_kernel<T, N><<<uint32_t(ceil_div(n, size_t(block.y) * kLookups)), block, 0, s>>>(              \
            static_cast<const T *>(table), table_stride, vocab, pieces, ids, wide, n, scale, static_cast<T *>(out), \
            out_stride);                                                                                         \
    }
    if (dt == GC_ROW_F32) { GC_BY_PIECE(float, m, GC_EMBED_CALL) }
    else if (dt == GC_ROW_BF16) { GC_BY_PIECE(__nv_bfloat16, m, GC_EMBED_CALL) }
    else { GC_BY_PIECE(__half, m, GC_EMBED_CALL) }
    return cudaGetLastError();
}

cudaError_t launch_embedding_grad(const void *g, size_t g_stride, gc_row_dtype gdt, const void *ids, bool wide,
                                  uint32_t n, uint32_t vocab, size_t width, float scale, void *dtable,
                                  size_t dtable_stride, gc_row_dtype odt, bool accumulate, uint8_t *ws, cudaStream_t s)
{
    const GradLayout l = grad_layout(n, vocab, width);
    uint2 *items[2] = {reinterpret_cast<uint2 *>(ws + l.items_a), reinterpret_cast<uint2 *>(ws + l.items_b)};
    uint32_t *table = reinterpret_cast<uint32_t *>(ws + l.table);
    uint8_t *seen = accumulate ? nullptr : ws + l.seen;
    float *edges = reinterpret_cast<float *>(ws + l.edges);
    const int bits = key_bits(vocab), passes = int(ceil_div(bits, 9)), digit = int(ceil_div(bits, passes));
    cudaError_t e = cudaSuccess;
    if (n > 0 && gcd::bin_chunks(n) == 1) {
        if (persistent_grid(reinterpret_cast<const void *>(token_sort_kernel), gcd::kBinThreads, sizeof(TokenSortSmem),
                            1) <= 0)
            return cudaErrorInvalidConfiguration;
        token_sort_kernel<<<1, gcd::kBinThreads, sizeof(TokenSortSmem), s>>>(
            ids, wide, n, vocab, uint32_t(digit), passes, items[passes & 1], seen);
        e = cudaGetLastError();
    } else {
        if (seen) e = cudaMemsetAsync(seen, 0, vocab, s);
        for (int p = 0; n > 0 && p < passes && e == cudaSuccess; ++p) {
            const TokenPass src{ids, items[p & 1], seen, p == 0, wide, vocab, uint32_t(p * digit), (1u << digit) - 1u};
            const TokenSink sink{src, items[(p & 1) ^ 1]};
            e = gcd::launch_bin_count(src, n, 1u << digit, table, s);
            if (e == cudaSuccess) e = gcd::launch_bin_place(src, sink, n, 1u << digit, 1u, table, s);
        }
    }
    if (e != cudaSuccess) return e;
    const uint2 *sorted = items[passes & 1];
    const GradOut out{dtable, dtable_stride, scale, accumulate, seen, vocab};
    if (gdt == GC_ROW_F32) return grad_rows<float, float>(sorted, n, g, g_stride, width, edges, out, s);
    if (gdt == GC_ROW_BF16)
        return odt == GC_ROW_F32 ? grad_rows<__nv_bfloat16, float>(sorted, n, g, g_stride, width, edges, out, s)
                                 : grad_rows<__nv_bfloat16, __nv_bfloat16>(sorted, n, g, g_stride, width, edges, out, s);
    return odt == GC_ROW_F32 ? grad_rows<__half, float>(sorted, n, g, g_stride, width, edges, out, s)
                             : grad_rows<__half, __half>(sorted, n, g, g_stride, width, edges, out, s);
}

}  // namespace gch
