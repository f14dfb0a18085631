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
#include <algorithm>

#include <math_constants.h>

#include "gc_binsort.cuh"
#include "gc_pipe.cuh"
#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr int kRowThreads = 256;
constexpr uint32_t kBlock = 32;     // sorted positions per block
constexpr int kLookups = 2;         // rows per thread of a lookup
constexpr size_t kZeroBytes = 32768;  // zeroed per CTA of the sums, about
// A bulk sum's CTA holds kBlock rows of up to this many bytes per row of
// threads, 64 KiB in all: three CTAs to an SM.
constexpr uint32_t kSliceBytes = 2048;
// Positions that one CTA sorts alone, the other CTAs zeroing the result
// meanwhile: 23 us for the gradient of 4096 tokens of 512 in a table of 32768,
// 31 us with the sort of more tokens, which takes over where both take as long.
constexpr uint32_t kSortAlone = 4096;
constexpr uint32_t kZeroCtas = 300;   // of them, two to an SM

// tx threads across a row's pieces, kRowThreads / tx rows.
dim3 row_block(size_t pieces)
{
    int tx = 32;
    while (tx < kRowThreads && size_t(tx) < pieces) tx <<= 1;
    return dim3(tx, kRowThreads / tx);
}

// A thread moves the same piece of kLookups rows, whose ids and then whose
// pieces are loaded together.  65536 of 128000 x 2048 bf16: 60 us, 86% of the
// copy rate.  Four rows a thread were 3% and eight 25% slower than two: the more
// rows an SM has under way, the worse HBM takes their mixture of reads and
// writes.
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
    constexpr int kCols = kNarrow<T, N>;
    for (uint32_t base = threadIdx.x; base < pieces; base += kCols * blockDim.x) {
        Piece<T, N> v[kLookups][kCols];
#pragma unroll
        for (int r = 0; r < kLookups; ++r)
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                const uint32_t c = base + q * blockDim.x;
                v[r][q] = zero_piece<T, N>();
                if (id[r] < vocab && c < pieces)
                    v[r][q] = load_piece<T, N>(table + size_t(id[r]) * table_stride + size_t(c) * N);
            }
#pragma unroll
        for (int r = 0; r < kLookups; ++r) {
            if (first + r >= n) break;
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                const uint32_t c = base + q * blockDim.x;
                if (c >= pieces) break;
                if (id[r] < vocab)  // zeros stay zeros whatever the scale
#pragma unroll
                    for (int k = 0; k < N; ++k) v[r][q].v[k] = row_from_float<T>(scale * row_to_float(v[r][q].v[k]));
                stream_piece<T, N>(out + size_t(first + r) * out_stride + size_t(c) * N, v[r][q]);
            }
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

// Rows [lo, hi) of the result, zeroed a warp to a row; with `seen`, only those
// of absent tokens.
struct ZeroRows {
    uint8_t *rows;
    size_t stride, bytes;  // of a row
    const uint8_t *seen;
    uint32_t lo, hi;
    __device__ __forceinline__ void run(uint32_t cta, uint32_t ctas) const
    {
        const uint32_t warps = blockDim.x * blockDim.y / 32, warp = (threadIdx.y * blockDim.x + threadIdx.x) / 32;
        const uint64_t first = lo + uint64_t(cta) * warps + warp;
        for (uint64_t v = first; v < hi; v += uint64_t(ctas) * warps) {
            if (seen != nullptr && seen[v]) continue;
            zero_row(rows + v * stride, bytes);
        }
    }
};

// A short sort by the first CTA, whose items stay in shared memory between
// the passes; the others zero the result.
struct TokenSortSmem {
    BinSmem bins;
    uint2 items[2][kSortAlone];
    uint32_t cnt[kBinWarps << 9];
};

__global__ void __launch_bounds__(kBinThreads)
token_sort_kernel(const void *ids, bool wide, uint32_t n, uint32_t vocab, uint32_t digit, int passes, uint2 *sorted,
                  uint32_t *header, ZeroRows zero)
{
    extern __shared__ __align__(16) uint8_t token_smem[];
    TokenSortSmem &sm = *reinterpret_cast<TokenSortSmem *>(token_smem);
    chain_start();
    if (blockIdx.x > 0) {
        zero.run(blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    if (threadIdx.x < kHeaderBytes / 4) header[threadIdx.x] = 0u;
    for (uint32_t i = threadIdx.x; i < n; i += kBinThreads) sm.items[0][i] = make_uint2(load_id(ids, wide, i, vocab), i);
    __syncthreads();
    for (int p = 0; p < passes; ++p) {
        const TokenPass src{nullptr, sm.items[p & 1], nullptr, false, wide, vocab, uint32_t(p) * digit,
                            (1u << digit) - 1u};
        const TokenSink sink{src, p + 1 < passes ? sm.items[(p & 1) ^ 1] : sorted};
        bin_place_chunk(src, sink, n, n, 1, 0, 1u << digit, 1u, nullptr, sm.cnt, sm.bins);
        __syncthreads();
    }
}

struct GradOut {
    void *rows;
    size_t stride;
    float scale;
    bool accumulate;
    uint32_t vocab;
};

// CTAs below `sums`: blocks of kBlock sorted positions, one to a row of
// threads, summed run by run.  edges: two rows per block, the sum of its
// first run where that began before the block, and of its last where that
// began in the block and goes on.  The other CTAs zero rows.
// The rows of the next kAhead positions, and what they are added to, are
// loaded while the ones before are summed.
template <class T, class O, int N, bool ADD>
__global__ void __launch_bounds__(kRowThreads, 4)
token_sums_kernel(const uint2 *__restrict__ sorted, uint32_t n, const T *__restrict__ g, size_t g_stride,
                  uint32_t width, float *__restrict__ edges, GradOut out, uint32_t parts, uint32_t sums, ZeroRows zero)
{
    O *rows = static_cast<O *>(out.rows);
    const uint32_t columns = blockDim.x * N;
    chain_start();
    chain_wait();
    if (blockIdx.x >= sums) {
        zero.run(blockIdx.x - sums, gridDim.x - sums);
        return;
    }
    // Keys of the block's positions between those of its neighbours, and the
    // positions; none: the end of the tokens in range.
    __shared__ uint32_t s_key[kRowThreads / 32][kBlock + 2], s_at[kRowThreads / 32][kBlock];
    // `parts` CTAs, neighbours in the grid, share a row
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
    constexpr int kAhead = (ADD ? 4 : 8) * (sizeof(T) * N <= 4 ? 2 : 1);
    Piece<T, N> x[kAhead];
    Piece<O, N> old[ADD ? kAhead : 1];
    auto load = [&](uint32_t at_j, int j) {
        const uint32_t k = at_j < kBlock ? key[at_j + 1] : none;
        if (k == none) return;
        x[j] = load_piece<T, N>(g + size_t(at[at_j]) * g_stride + c);
        if (ADD && key[at_j + 2] != k) old[ADD ? j : 0] = load_piece<O, N>(rows + size_t(k) * out.stride + c);
    };
    Piece<float, N> sum{};
    bool began = key[0] != key[1];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load(j, j);
    for (uint32_t base = 0; base < kBlock; base += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t k = key[base + j + 1];
            if (k == none) return;
#pragma unroll
            for (int e = 0; e < N; ++e) sum.v[e] += row_to_float(x[j].v[e]);
            const bool ends = key[base + j + 2] != k;
            if (ends && began) {
                Piece<O, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float r = out.scale * sum.v[e];
                    o.v[e] = row_from_float<O>(ADD ? r + row_to_float(old[ADD ? j : 0].v[e]) : r);
                }
                store_piece<O, N>(rows + size_t(k) * out.stride + c, o);
            } else if (ends || base + j + 1 == kBlock) {
                store_piece<float, N>(edges + (size_t(block) * 2 + (began ? 1 : 0)) * width + c, sum);
            }
            if (ends) {
                sum = Piece<float, N>{};
                began = true;
            }
            load(base + kAhead + j, j);
        }
    }
}

// Until a block's copies have arrived.  Past timeout_ns the wait is recorded
// as GC_ERR_TIMEOUT, and past twice that it is given up: false.
__device__ __forceinline__ bool staged_wait(uint64_t *bar, uint8_t *ws, uint64_t timeout_ns)
{
    if (mbar_try_wait(bar, 0u)) return true;
    const uint64_t t0 = global_timer_ns();
    for (bool late = false; !mbar_try_wait(bar, 0u);) {
        const uint64_t waited = global_timer_ns() - t0;
        if (late && waited > 2 * timeout_ns) return false;
        if (!late && waited > timeout_ns) {
            record_error(ws, kTimeoutCode, 0xffffffffu);
            late = true;
        }
    }
    return true;
}

// The same where rows can be copied in bulk (16-byte aligned): the block's
// rows are copied into shared memory by the TMA unit, all at once, so that
// the whole block is in flight without registers; and the rows to be added to
// are fetched to L2.  blockDim.x threads, N elements each, to a slice.  The
// gradient of 32768 tokens of 128000 x 2048 bf16 takes 203 us by these kernels
// and 231 by the one above (193 since the join takes eight blocks a CTA), of
// 4096 x 512 23 and 29; 1.05 GB of it is the table, written at 6.9 TB/s.  Where
// the copies do not arrive the block's sums are NaN.  `missing`: bytes waited
// for that nobody copies (0 but in a test).
template <class T, class O, int N, bool ADD>
__global__ void __launch_bounds__(kRowThreads)
token_bulk_sums_kernel(const uint2 *__restrict__ sorted, uint32_t n, const T *__restrict__ g, size_t g_stride,
                       uint32_t width, float *__restrict__ edges, GradOut out, uint32_t parts, uint8_t *ws,
                       uint64_t timeout_ns, uint32_t missing, uint32_t sums, ZeroRows zero)
{
    chain_start();
    chain_wait();
    if (blockIdx.x >= sums) {
        zero.run(blockIdx.x - sums, gridDim.x - sums);
        return;
    }
    extern __shared__ __align__(16) uint8_t slice_smem[];
    __shared__ uint32_t s_key[kRowThreads / 32][kBlock + 2], s_at[kRowThreads / 32][kBlock];
    __shared__ uint64_t s_bar[kRowThreads / 32];
    O *rows = static_cast<O *>(out.rows);
    const uint32_t columns = blockDim.x * N, lane = threadIdx.x & 31;
    const uint32_t block = blockIdx.x / parts * blockDim.y + threadIdx.y, first = block * kBlock;
    const uint32_t none = out.vocab;
    uint32_t *key = s_key[threadIdx.y], *at = s_at[threadIdx.y];
    const uint32_t c0 = (blockIdx.x % parts) * columns, here = min(columns, width - c0);
    T *slice = reinterpret_cast<T *>(slice_smem) + size_t(threadIdx.y) * kBlock * columns;
    for (uint32_t j = threadIdx.x; j < kBlock + 2; j += blockDim.x) {
        const uint32_t i = first + j - 1;  // wraps before the first
        const uint2 item = i < n ? sorted[i] : make_uint2(none, 0u);
        key[j] = item.x;
        if (j >= 1 && j <= kBlock) at[j - 1] = item.y;
    }
    if (threadIdx.x == 0) {
        mbar_init(&s_bar[threadIdx.y], 1u);
        fence_barrier_init();
    }
    __syncthreads();
    if (key[1] == none) return;
    if (threadIdx.x < 32) {
        // Lane j copies row j; the tokens in range come first.
        const uint32_t k = key[lane + 1];
        const uint32_t rows_in = uint32_t(__popc(__ballot_sync(kFullMask, k != none)));
        if (lane == 0) mbar_arrive_expect_tx(&s_bar[threadIdx.y], rows_in * here * uint32_t(sizeof(T)) + missing);
        __syncwarp();
        if (k != none) {
            bulk_load(slice + size_t(lane) * columns, g + size_t(at[lane]) * g_stride + c0, here * uint32_t(sizeof(T)),
                      &s_bar[threadIdx.y]);
            if (ADD && key[lane + 2] != k) {
                const O *old = rows + size_t(k) * out.stride + c0;
                for (uint32_t e = 0; e < here; e += 128 / sizeof(O)) asm volatile("prefetch.global.L2 [%0];" ::"l"(old + e));
            }
        }
    }
    const bool arrived = staged_wait(&s_bar[threadIdx.y], ws, timeout_ns);
    const uint32_t c = threadIdx.x * N;
    if (c >= here) return;
    if (!arrived) {
        Piece<T, N> nan;
#pragma unroll
        for (int e = 0; e < N; ++e) nan.v[e] = row_from_float<T>(CUDART_NAN_F);
        for (uint32_t j = 0; j < kBlock; ++j) store_piece<T, N>(slice + size_t(j) * columns + c, nan);
    }
    Piece<float, N> sum{};
    bool began = key[0] != key[1];
    constexpr int kAhead = 4;
    for (uint32_t base = 0; base < kBlock; base += kAhead) {
        Piece<O, N> old[ADD ? kAhead : 1];
        if (ADD)
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (key[base + j + 1] != none && key[base + j + 2] != key[base + j + 1])
                    old[ADD ? j : 0] = load_piece<O, N>(rows + size_t(key[base + j + 1]) * out.stride + c0 + c);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t k = key[base + j + 1];
            if (k == none) return;
            const Piece<T, N> x = load_piece<T, N>(slice + size_t(base + j) * columns + c);
#pragma unroll
            for (int e = 0; e < N; ++e) sum.v[e] += row_to_float(x.v[e]);
            const bool ends = key[base + j + 2] != k;
            if (ends && began) {
                Piece<O, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float r = out.scale * sum.v[e];
                    o.v[e] = row_from_float<O>(ADD ? r + row_to_float(old[ADD ? j : 0].v[e]) : r);
                }
                store_piece<O, N>(rows + size_t(k) * out.stride + c0 + c, o);
            } else if (ends || base + j + 1 == kBlock) {
                store_piece<float, N>(edges + (size_t(block) * 2 + (began ? 1 : 0)) * width + c0 + c, sum);
            }
            if (ends) {
                sum = Piece<float, N>{};
                began = true;
            }
        }
    }
}

// Tokens whose run crosses blocks: the block in which it began adds up its
// parts.  A CTA takes kJoiners blocks and 32 pieces of a row, a warp to a
// block; a run that reaches more than kAhead further blocks is left to all
// warps, which take a share of them each and add the shares in order.
constexpr int kJoiners = 8;

template <class O, int N>
__global__ void __launch_bounds__(32 * kJoiners)
token_join_kernel(const uint2 *__restrict__ sorted, uint32_t n, uint32_t width, const float *__restrict__ edges,
                  GradOut out, uint32_t parts)
{
    constexpr uint32_t kAhead = 8;
    __shared__ Piece<float, N> s_sum[kJoiners][32];
    __shared__ uint32_t s_more[kJoiners], s_key[kJoiners];
    chain_wait();
    const uint32_t lane = threadIdx.x, warp = threadIdx.y;
    const uint32_t group = blockIdx.x / parts * kJoiners, block = group + warp;
    const uint32_t c = (blockIdx.x % parts) * 32 * N + lane * N;
    const uint32_t blocks = (n + kBlock - 1) / kBlock;
    // Blocks b + lo + 1 to b + hi of the run that began in block b.
    auto add = [&](Piece<float, N> &sum, uint32_t b, uint32_t lo, uint32_t hi) {
        const float *e = edges + (size_t(b) + lo + 1) * 2 * width + c;
        for (uint32_t i = lo; i < hi; i += kAhead) {
            Piece<float, N> x[kAhead];
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                x[j] = Piece<float, N>{};
                if (i + j < hi) x[j] = load_piece<float, N>(e + size_t(j) * 2 * width);
            }
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j)
#pragma unroll
                for (int k = 0; k < N; ++k) sum.v[k] += x[j].v[k];
            e += size_t(kAhead) * 2 * width;
        }
    };
    auto put = [&](uint32_t key, const Piece<float, N> &sum) {
        O *dst = static_cast<O *>(out.rows) + size_t(key) * out.stride + c;
        Piece<O, N> o;
        if (out.accumulate) o = load_piece<O, N>(dst);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float r = out.scale * sum.v[k];
            o.v[k] = row_from_float<O>(out.accumulate ? r + row_to_float(o.v[k]) : r);
        }
        store_piece<O, N>(dst, o);
    };
    uint32_t more = 0u;
    if (block + 1 < blocks) {
        const uint32_t first = block * kBlock, next = first + kBlock;
        const uint32_t key = sorted[next - 1].x, after = sorted[next].x, before = first > 0 ? sorted[first - 1].x : ~0u;
        if (key < out.vocab && after == key && before != key) {
            // The blocks whose first key is it: the run reaches them.
            more = 1;
            for (bool on = true; on;) {
                const uint32_t b = block + more + 1 + lane;
                const uint32_t same =
                    __ballot_sync(kFullMask, b < blocks && sorted[size_t(min(b, blocks - 1)) * kBlock].x == key);
                more += same == kFullMask ? 32u : uint32_t(__ffs(~same) - 1);
                on = same == kFullMask;
            }
            if (more <= kAhead && c < width) {
                Piece<float, N> sum = load_piece<float, N>(edges + (size_t(block) * 2 + 1) * width + c);
                add(sum, block, 0, more);
                put(key, sum);
            }
            if (lane == 0) s_key[warp] = key;
        }
    }
    if (lane == 0) s_more[warp] = more > kAhead ? more : 0u;
    __syncthreads();
    for (uint32_t w = 0; w < kJoiners; ++w) {
        const uint32_t far = s_more[w];
        if (far == 0u) continue;  // the same for all
        const uint32_t b = group + w, per = (far + kJoiners - 1) / kJoiners;
        Piece<float, N> sum{};
        if (c < width) {
            if (warp == 0) sum = load_piece<float, N>(edges + (size_t(b) * 2 + 1) * width + c);
            add(sum, b, min(far, warp * per), min(far, (warp + 1) * per));
        }
        s_sum[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && c < width) {
            for (int j = 1; j < kJoiners; ++j)
#pragma unroll
                for (int k = 0; k < N; ++k) sum.v[k] += s_sum[j][lane].v[k];
            put(s_key[w], sum);
        }
        __syncthreads();
    }
}

int key_bits(size_t vocab)
{
    int bits = 1;
    while ((size_t(vocab) >> bits) != 0) ++bits;
    return bits;
}

// The workspace starts with the library's header, of which only the error
// word is used; `seen` follows, so that one clear serves both.
struct GradLayout {
    size_t seen, items_a, items_b, table, edges, total;
};

GradLayout grad_layout(size_t n, size_t vocab, size_t width)
{
    GradLayout l{};
    const size_t items = gch::align_up(8 * n, 256);
    l.seen = kHeaderBytes;
    l.items_a = l.seen + gch::align_up(vocab, 256);
    l.items_b = l.items_a + items;
    l.table = l.items_b + items;
    l.edges = l.table + gch::align_up(bin_table_bytes(n, 512), 256);
    l.total = l.edges + gch::align_up(gch::ceil_div(n, size_t(kBlock)) * 2 * width * 4, 256) + 256;
    return l;
}

// CTAs for the rest of the rows to zero.
uint32_t zero_ctas(const ZeroRows &z)
{
    const size_t rows = z.hi - z.lo, per = kZeroBytes / z.bytes < 8 ? 8 : kZeroBytes / z.bytes;
    return uint32_t(gch::ceil_div(rows, per));
}

template <class T, class O, int N>
cudaError_t run_grad_rows(const uint2 *sorted, uint32_t n, const void *g, size_t g_stride, size_t width, float *edges,
                          const GradOut &out, const ZeroRows &zero, uint8_t *ws, const gch::StagedWait &wait,
                          cudaStream_t s)
{
    const uint32_t blocks = uint32_t(gch::ceil_div(n, kBlock)), zeros = zero_ctas(zero);
    // Bulk copies need 16-byte aligned rows; a slice narrower than a warp's
    // pieces is not worth one.
    const bool bulk = ((uintptr_t(g) | g_stride * sizeof(T) | width * sizeof(T)) & 15u) == 0 && width / N >= 32;
    dim3 threads = row_block(width / N);
    if (bulk) {
        const uint32_t most = kSliceBytes / (N * sizeof(T));
        if (threads.x > most) threads.x = most;
        threads.y = std::min(kRowThreads / threads.x, kSliceBytes / uint32_t(threads.x * N * sizeof(T)));
    }
    const size_t parts = gch::ceil_div(width / N, threads.x);
    const size_t sums = gch::ceil_div(blocks, threads.y) * parts;
    const size_t joins = blocks > 1 ? gch::ceil_div(blocks - 1, kJoiners) * gch::ceil_div(width / N, 32) : 0;
    if (sums + zeros > 0x7fffffffu || joins > 0x7fffffffu) return cudaErrorInvalidConfiguration;
    if (n == 0) {
        // Only zeros, after the clear, which is no kernel to chain to.
        if (zeros > 0)
            token_sums_kernel<T, O, N, false><<<zeros, threads, 0, s>>>(sorted, n, static_cast<const T *>(g), g_stride,
                                                                       uint32_t(width), edges, out, uint32_t(parts), 0u,
                                                                       zero);
        return cudaGetLastError();
    }
    if (bulk) {
        auto kernel = out.accumulate ? token_bulk_sums_kernel<T, O, N, true> : token_bulk_sums_kernel<T, O, N, false>;
        const size_t smem = size_t(threads.x) * N * sizeof(T) * kBlock * threads.y;
        // Raises the kernel's shared-memory limit, once per device.
        if (gch::persistent_grid(reinterpret_cast<const void *>(kernel), kRowThreads, size_t(kSliceBytes) * kBlock, 1) <= 0)
            return cudaErrorInvalidConfiguration;
        const cudaError_t e = gch::launch_next(kernel, dim3(uint32_t(sums + zeros)), threads, smem, s, sorted, n,
                                               static_cast<const T *>(g), g_stride, uint32_t(width), edges, out,
                                               uint32_t(parts), ws, wait.timeout_ns, wait.missing, uint32_t(sums), zero);
        if (e != cudaSuccess) return e;
    } else {
        auto kernel = out.accumulate ? token_sums_kernel<T, O, N, true> : token_sums_kernel<T, O, N, false>;
        const cudaError_t e = gch::launch_next(kernel, dim3(uint32_t(sums + zeros)), threads, 0, s, sorted, n,
                                               static_cast<const T *>(g), g_stride, uint32_t(width), edges, out,
                                               uint32_t(parts), uint32_t(sums), zero);
        if (e != cudaSuccess) return e;
    }
    if (joins > 0)
        return gch::launch_next(token_join_kernel<O, N>, dim3(uint32_t(joins)), dim3(32, kJoiners), 0, s, sorted, n,
                                uint32_t(width), static_cast<const float *>(edges), out,
                                uint32_t(gch::ceil_div(width / N, 32)));
    return cudaSuccess;
}

// Pieces of N elements, N a power of two that both rows allow and that fills
// 16 bytes of the result at most.
#define GC_GRAD_CALL(T, O, N) return run_grad_rows<T, O, N>(sorted, n_, g, g_stride, width, edges, out, zero, ws, wait, s)
template <class T, class O>
cudaError_t grad_rows(const uint2 *sorted, uint32_t n_, const void *g, size_t g_stride, size_t width, float *edges,
                      const GradOut &out, const ZeroRows &zero, uint8_t *ws, const gch::StagedWait &wait, cudaStream_t s)
{
    const int in = gch::piece_elems(uint64_t(uintptr_t(g)) | sizeof(T) * (g_stride | width), sizeof(T));
    const int to = gch::piece_elems(uint64_t(uintptr_t(out.rows)) | sizeof(O) * (out.stride | width), sizeof(O));
    switch (in < to ? in : to) {
    case 1: GC_GRAD_CALL(T, O, 1);
    case 2: GC_GRAD_CALL(T, O, 2);
    case 4: GC_GRAD_CALL(T, O, 4);
    default: GC_GRAD_CALL(T, O, 16 / int(sizeof(O)));
    }
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
                                  size_t dtable_stride, gc_row_dtype odt, bool accumulate, uint8_t *ws, cudaStream_t s,
                                  const StagedWait &wait)
{
    const GradLayout l = grad_layout(n, vocab, width);
    uint2 *items[2] = {reinterpret_cast<uint2 *>(ws + l.items_a), reinterpret_cast<uint2 *>(ws + l.items_b)};
    uint32_t *table = reinterpret_cast<uint32_t *>(ws + l.table);
    uint8_t *seen = accumulate ? nullptr : ws + l.seen;
    float *edges = reinterpret_cast<float *>(ws + l.edges);
    const int bits = key_bits(vocab), passes = int(ceil_div(bits, 9)), digit = int(ceil_div(bits, passes));
    const size_t elem = odt == GC_ROW_F32 ? 4 : 2;
    ZeroRows zero{static_cast<uint8_t *>(dtable), dtable_stride * elem, width * elem, seen, 0u, accumulate ? 0u : vocab};
    cudaError_t e = cudaSuccess;
    if (vocab == 0) return cudaMemsetAsync(ws, 0, kHeaderBytes, s);  // no row, and no error
    if (n > 0 && n <= kSortAlone) {
        // Everything is zeroed here, before any row is written.
        if (persistent_grid(reinterpret_cast<const void *>(token_sort_kernel), gcd::kBinThreads, sizeof(TokenSortSmem),
                            1) <= 0)
            return cudaErrorInvalidConfiguration;
        zero.seen = nullptr;
        const uint32_t others = std::min(zero_ctas(zero), kZeroCtas);
        token_sort_kernel<<<1 + others, gcd::kBinThreads, sizeof(TokenSortSmem), s>>>(
            ids, wide, n, vocab, uint32_t(digit), passes, items[passes & 1], reinterpret_cast<uint32_t *>(ws), zero);
        zero.lo = zero.hi;
        e = cudaGetLastError();
    } else {
        e = cudaMemsetAsync(ws, 0, accumulate ? size_t(kHeaderBytes) : l.seen + vocab, s);
        for (int p = 0; n > 0 && p < passes && e == cudaSuccess; ++p) {
            const TokenPass src{ids, items[p & 1], seen, p == 0, wide, vocab, uint32_t(p * digit), (1u << digit) - 1u};
            const TokenSink sink{src, items[(p & 1) ^ 1]};
            e = gcd::launch_bin_count(src, n, 1u << digit, table, s, p > 0);
            if (e == cudaSuccess) e = gcd::launch_bin_place(src, sink, n, 1u << digit, 1u, table, s);
        }
    }
    if (e != cudaSuccess) return e;
    const uint2 *sorted = items[passes & 1];
    const GradOut out{dtable, dtable_stride, scale, accumulate, vocab};
    if (gdt == GC_ROW_F32) return grad_rows<float, float>(sorted, n, g, g_stride, width, edges, out, zero, ws, wait, s);
    if (gdt == GC_ROW_BF16)
        return odt == GC_ROW_F32
                   ? grad_rows<__nv_bfloat16, float>(sorted, n, g, g_stride, width, edges, out, zero, ws, wait, s)
                   : grad_rows<__nv_bfloat16, __nv_bfloat16>(sorted, n, g, g_stride, width, edges, out, zero, ws, wait, s);
    return odt == GC_ROW_F32 ? grad_rows<__half, float>(sorted, n, g, g_stride, width, edges, out, zero, ws, wait, s)
                             : grad_rows<__half, __half>(sorted, n, g, g_stride, width, edges, out, zero, ws, wait, s);
}

}  // namespace gch
