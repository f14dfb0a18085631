// experts.cu -- tokens sorted by expert and back (gc_expert_dispatch,
// gc_expert_combine, gc_expert_combine_grad).
//
// The plan is a stable partition of the tokens * topk pairs into one bin per
// expert (gc_binsort.cuh); the rest moves rows: one row per pair out, a
// weighted sum of topk rows per token back, and for the gradient one scaled
// row and one dot product per pair.  Plans wait for memory (11 us for 131072
// pairs, three kernels); the row kernels are bound by HBM traffic, and each
// works token by token, so that a token's row is read once and the k rows of
// its experts are the only ones touched at random, whole rows at a time.
#include "gc_binsort.cuh"
#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

struct ExpertSource {
    const void *ids;
    bool wide;
    uint32_t experts;
    __device__ __forceinline__ uint32_t bin(uint32_t i) const { return load_id(ids, wide, i, experts); }
    __device__ __forceinline__ void visit(uint32_t) const {}
};

struct ExpertSink {
    int32_t *offsets, *counts, *slots, *pairs;
    uint32_t experts;
    __device__ __forceinline__ void start(uint32_t b, uint32_t start, uint32_t count) const
    {
        offsets[b] = int32_t(start);
        counts[b] = int32_t(count);
    }
    __device__ __forceinline__ void end(uint32_t total) const { offsets[experts] = int32_t(total); }
    __device__ __forceinline__ void place(uint32_t p, uint32_t row) const
    {
        slots[p] = int32_t(row);
        pairs[row] = int32_t(p);
    }
    __device__ __forceinline__ void drop(uint32_t p) const { slots[p] = -1; }
};

// Threads of a row kernel: `tx` across one row's pieces, kRowThreads / tx rows.
constexpr int kRowThreads = 256;

dim3 row_block(size_t pieces)
{
    int tx = 32;
    while (tx < kRowThreads && size_t(tx) < pieces) tx <<= 1;
    return dim3(tx, kRowThreads / tx);
}

// Rows without a pair: -1 in pairs and zeros.  One warp takes kPadRows rows,
// each lane looks one up in the experts' blocks.
constexpr uint32_t kPadRows = 16;

__device__ __forceinline__ void expert_pad_rows(uint32_t first, uint32_t rows, uint32_t experts,
                                                const int32_t *__restrict__ offsets,
                                                const int32_t *__restrict__ counts, int32_t *__restrict__ pairs,
                                                uint8_t *__restrict__ out, size_t stride_bytes, size_t row_bytes)
{
    const uint32_t lane = threadIdx.x & 31, r = first + lane;
    bool pad = false;
    if (lane < kPadRows && r < rows) {
        pad = r >= uint32_t(offsets[experts]);
        if (!pad) {
            // the last block that starts at or before r, which is not an empty one
            uint32_t lo = 0, hi = experts;
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                if (uint32_t(offsets[mid]) <= r) lo = mid;
                else hi = mid;
            }
            pad = r - uint32_t(offsets[lo]) >= uint32_t(counts[lo]);
        }
        if (pad) pairs[r] = -1;
    }
    uint32_t left = __ballot_sync(0xffffffffu, pad);
    if (out == nullptr) return;
    for (; left; left &= left - 1) zero_row(out + size_t(first + __ffs(left) - 1) * stride_bytes, row_bytes);
}

// One token's row to its slots: read once, kSpread pieces per thread at a
// time, and written up to topk times.  Against gathering by destination row,
// which reads every token's row topk times (from L2 at best): 16384 x 8 pairs
// of 2048 bf16, 205 -> 126 us with the plan, 100 us of it the bytes at the copy
// rate.  Rows of odd width move element by element, and are latency-bound: 1531
// x 3 of 1001 float16 37 us with one element per thread at a time, 20 with four.
constexpr int kSpread = 4;

template <class E, int N>
__device__ __forceinline__ void expert_spread_row(const E *__restrict__ src, const uint32_t *slots, uint32_t topk,
                                                  uint32_t rows, E *__restrict__ out, size_t out_stride,
                                                  uint32_t pieces)
{
    for (uint32_t base = threadIdx.x; base < pieces; base += kSpread * blockDim.x) {
        Piece<E, N> v[kSpread];
#pragma unroll
        for (int q = 0; q < kSpread; ++q) {
            const uint32_t c = base + q * blockDim.x;
            if (c < pieces) v[q] = load_piece<E, N>(src + size_t(c) * N);
        }
        for (uint32_t j = 0; j < topk; ++j) {
            if (slots[j] >= rows) continue;
            E *dst = out + size_t(slots[j]) * out_stride;
#pragma unroll
            for (int q = 0; q < kSpread; ++q) {
                const uint32_t c = base + q * blockDim.x;
                if (c < pieces) stream_piece<E, N>(dst + size_t(c) * N, v[q]);
            }
        }
    }
}

// E: an integer of the element's size.  CTAs below `spread` move tokens, one
// to a row of threads; the others look for rows without a pair.
template <class E, int N>
__global__ void __launch_bounds__(kRowThreads)
expert_rows_kernel(const E *__restrict__ x, size_t x_stride, uint32_t tokens, uint32_t topk, uint32_t experts,
                   const int32_t *__restrict__ offsets, const int32_t *__restrict__ counts,
                   const int32_t *__restrict__ slots, int32_t *__restrict__ pairs, uint32_t rows,
                   E *__restrict__ out, size_t out_stride, uint32_t pieces, uint32_t spread)
{
    chain_wait();
    if (blockIdx.x >= spread) {
        const uint32_t warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5;
        const uint64_t first = (uint64_t(blockIdx.x - spread) * (kRowThreads / 32) + warp) * kPadRows;
        if (first < rows)
            expert_pad_rows(uint32_t(first), rows, experts, offsets, counts, pairs, reinterpret_cast<uint8_t *>(out),
                            out_stride * sizeof(E), size_t(pieces) * N * sizeof(E));
        return;
    }
    __shared__ uint32_t s_slots[kRowThreads / 32][GC_MAX_TOPK];
    const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t < tokens && threadIdx.x < topk) {
        // 32 threads at least to a row, 64 choices at most
        s_slots[threadIdx.y][threadIdx.x] = uint32_t(slots[size_t(t) * topk + threadIdx.x]);
        if (threadIdx.x + 32 < topk && blockDim.x == 32)
            s_slots[threadIdx.y][threadIdx.x + 32] = uint32_t(slots[size_t(t) * topk + threadIdx.x + 32]);
    }
    __syncthreads();
    if (t < tokens)
        expert_spread_row<E, N>(x + size_t(t) * x_stride, s_slots[threadIdx.y], topk, rows, out, out_stride, pieces);
}

// The whole dispatch of up to kSmallPairs pairs in one launch: every CTA counts
// all pairs itself.  CTAs below tokens move one token each, the others look for
// rows without a pair.  Rows of 2048 bf16, this against the three kernels for
// more pairs: 64 pairs 3.1 against 5.4 us, 2048 pairs 5.0 against 8.7, 4096
// pairs 8.1 against 9.9, 8192 pairs 17.9 against 12.4.
constexpr uint32_t kSmallPairs = 4096;

template <class E, int N>
__global__ void __launch_bounds__(kRowThreads)
expert_small_kernel(ExpertSource src, ExpertSink sink, uint32_t npairs, uint32_t topk, uint32_t align,
                    const E *__restrict__ x, size_t x_stride, uint32_t rows, E *__restrict__ out, size_t out_stride,
                    uint32_t pieces)
{
    __shared__ uint32_t s_ids[kSmallPairs];
    __shared__ int32_t s_counts[GC_MAX_EXPERTS], s_offsets[GC_MAX_EXPERTS + 1];
    __shared__ uint32_t s_slots[GC_MAX_TOPK], s_warp[kRowThreads / 32];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, experts = src.experts;
    for (uint32_t e = tid; e < experts; e += kRowThreads) s_counts[e] = 0;
    __syncthreads();
    for (uint32_t p = tid; p < npairs; p += kRowThreads) {
        const uint32_t e = src.bin(p);
        s_ids[p] = e;
        if (e < experts) atomicAdd(&s_counts[e], 1);
    }
    __syncthreads();
    const uint32_t per = (experts + kRowThreads - 1) / kRowThreads;
    const uint32_t lo = min(experts, tid * per), hi = min(experts, lo + per);
    uint32_t sum = 0u, total;
    for (uint32_t e = lo; e < hi; ++e) sum += (uint32_t(s_counts[e]) + align - 1u) / align * align;
    uint32_t start = bin_block_scan<kRowThreads>(sum, s_warp, total);
    for (uint32_t e = lo; e < hi; ++e) {
        s_offsets[e] = int32_t(start);
        if (blockIdx.x == 0) sink.start(e, start, uint32_t(s_counts[e]));
        start += (uint32_t(s_counts[e]) + align - 1u) / align * align;
    }
    if (tid == 0) {
        s_offsets[experts] = int32_t(total);
        if (blockIdx.x == 0) sink.end(total);
    }
    __syncthreads();
    const uint32_t t = blockIdx.x, tokens = npairs / topk;
    if (t >= tokens) {
        const uint32_t first = ((t - tokens) * (kRowThreads / 32) + warp) * kPadRows;
        if (first < rows)
            expert_pad_rows(first, rows, experts, s_offsets, s_counts, sink.pairs, reinterpret_cast<uint8_t *>(out),
                            out_stride * sizeof(E), size_t(pieces) * N * sizeof(E));
        return;
    }
    // A warp per choice: the earlier pairs of the same expert.
    for (uint32_t j = warp; j < topk; j += kRowThreads / 32) {
        const uint32_t p = t * topk + j, e = s_ids[p];
        uint32_t rank = 0u;
        for (uint32_t q = lane; q < p; q += 32) rank += s_ids[q] == e;
        rank = __reduce_add_sync(0xffffffffu, rank);
        const uint32_t row = e < experts ? uint32_t(s_offsets[e]) + rank : ~0u;
        if (lane == 0) {
            s_slots[j] = row;
            if (e < experts) sink.place(p, row);
            else sink.drop(p);
        }
    }
    __syncthreads();
    if (out != nullptr)
        expert_spread_row<E, N>(x + size_t(t) * x_stride, s_slots, topk, rows, out, out_stride, pieces);
}

// The rows of kAhead choices are loaded together; sums in float32 in the order
// of the choices.  16384 x 8 pairs of 2048 bf16: 109 us, 83% of the copy rate
// (604 MB); with 8 choices at a time 160 us and with 2 at six CTAs per SM 190,
// for want of registers.
constexpr int kAhead = 4;

template <class T, int N>
__global__ void __launch_bounds__(kRowThreads, 4)
expert_combine_kernel(const T *__restrict__ y, size_t y_stride, uint32_t rows, const int32_t *__restrict__ slots,
                      const float *__restrict__ weights, uint32_t tokens, uint32_t topk, uint32_t pieces,
                      T *__restrict__ out, size_t out_stride)
{
    constexpr int kCols = sizeof(T) * N >= 8 ? 1 : kNarrow<T, N>;  // at 8 bytes two cost more registers than they give
    const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    for (uint32_t first = threadIdx.x; first < pieces; first += kCols * blockDim.x) {
        float acc[kCols][N] = {};
        for (uint32_t base = 0; base < topk; base += kAhead) {
            uint32_t slot[kAhead];
            float w[kAhead];
            Piece<T, N> v[kAhead][kCols];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const uint64_t p = uint64_t(t) * topk + base + j;
                slot[j] = base + j < topk ? uint32_t(slots[p]) : ~0u;
                w[j] = weights && base + j < topk ? weights[p] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (slot[j] < rows)
#pragma unroll
                    for (int q = 0; q < kCols; ++q) {
                        const uint32_t c = first + q * blockDim.x;
                        if (c < pieces) v[j][q] = load_piece<T, N>(y + size_t(slot[j]) * y_stride + size_t(c) * N);
                    }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (slot[j] < rows)
#pragma unroll
                    for (int q = 0; q < kCols; ++q)
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[q][i] = fmaf(w[j], row_to_float(v[j][q].v[i]), acc[q][i]);
        }
#pragma unroll
        for (int q = 0; q < kCols; ++q) {
            const uint32_t c = first + q * blockDim.x;
            if (c >= pieces) break;
            Piece<T, N> o;
#pragma unroll
            for (int i = 0; i < N; ++i) o.v[i] = row_from_float<T>(acc[q][i]);
            store_piece<T, N>(out + size_t(t) * out_stride + size_t(c) * N, o);
        }
    }
}

// One warp per pair: the scaled gradient row and the dot product; then one
// warp per row without a pair: zeros.  A token's pairs are neighbouring warps,
// so its gradient row comes from HBM once.  8192 x 8 pairs of 4096 bf16: 182 us,
// 93% of the copy rate.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads)
expert_combine_grad_kernel(const T *__restrict__ g, size_t g_stride, const T *__restrict__ y, size_t y_stride,
                           uint32_t rows, const int32_t *__restrict__ slots, const int32_t *__restrict__ pairs,
                           const float *__restrict__ weights, uint32_t npairs, uint32_t topk, uint32_t pieces,
                           T *__restrict__ dy, size_t dy_stride, float *__restrict__ dweights)
{
    const uint64_t unit = uint64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const uint32_t lane = threadIdx.x & 31;
    if (unit < npairs) {
        const uint32_t p = uint32_t(unit);
        const uint32_t slot = uint32_t(slots[p]);
        float dot = 0.0f;
        if (slot < rows) {
            const float w = weights ? weights[p] : 1.0f;
            const T *gr = g + size_t(p / topk) * g_stride;
            constexpr int kCols = kNarrow<T, N>;
            for (uint32_t first = lane; first < pieces; first += 32 * kCols) {
                // Narrow pieces of both rows are loaded together; 16-byte ones
                // of y after the store, which is the faster order for them (98
                // against 106 us for 8192 x 8 pairs of 2048 bf16).
                Piece<T, N> a[kCols], b[kCols];
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    const uint32_t c = first + 32 * q;
                    if (c >= pieces) break;
                    a[q] = load_piece<T, N>(gr + size_t(c) * N);
                    if (kCols > 1 && dweights) b[q] = load_piece<T, N>(y + size_t(slot) * y_stride + size_t(c) * N);
                }
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    const uint32_t c = first + 32 * q;
                    if (c >= pieces) break;
                    Piece<T, N> o;
#pragma unroll
                    for (int i = 0; i < N; ++i) o.v[i] = row_from_float<T>(w * row_to_float(a[q].v[i]));
                    stream_piece<T, N>(dy + size_t(slot) * dy_stride + size_t(c) * N, o);
                    if (dweights) {
                        if (kCols == 1) b[q] = load_piece<T, N>(y + size_t(slot) * y_stride + size_t(c) * N);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot = fmaf(row_to_float(a[q].v[i]), row_to_float(b[q].v[i]), dot);
                    }
                }
            }
        }
        if (dweights) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (lane == 0) dweights[p] = dot;
        }
    } else if (unit - npairs < rows) {
        const uint32_t r = uint32_t(unit - npairs);
        if (uint32_t(pairs[r]) < npairs) return;
        for (uint32_t c = lane; c < pieces; c += 32)
            store_piece<T, N>(dy + size_t(r) * dy_stride + size_t(c) * N, zero_piece<T, N>());
    }
}

template <class T, int N>
void run_combine(const void *y, size_t y_stride, uint32_t rows, const int32_t *slots, const float *weights,
                 uint32_t tokens, uint32_t topk, size_t width, void *out, size_t out_stride, cudaStream_t s)
{
    const uint32_t pieces = uint32_t(width / N);
    const dim3 block = row_block(pieces);
    expert_combine_kernel<T, N><<<uint32_t(gch::ceil_div(tokens, block.y)), block, 0, s>>>(
        static_cast<const T *>(y), y_stride, rows, slots, weights, tokens, topk, pieces, static_cast<T *>(out),
        out_stride);
}

template <class T, int N>
void run_combine_grad(const void *g, size_t g_stride, const void *y, size_t y_stride, uint32_t rows,
                      const int32_t *slots, const int32_t *pairs, const float *weights, uint32_t npairs,
                      uint32_t topk, size_t width, void *dy, size_t dy_stride, float *dweights, cudaStream_t s)
{
    const uint64_t units = uint64_t(npairs) + rows;
    expert_combine_grad_kernel<T, N><<<uint32_t(gch::ceil_div(units, kRowThreads / 32)), kRowThreads, 0, s>>>(
        static_cast<const T *>(g), g_stride, static_cast<const T *>(y), y_stride, rows, slots, pairs, weights,
        npairs, topk, uint32_t(width / N), static_cast<T *>(dy), dy_stride, dweights);
}

template <class E, int N>
void run_rows(const void *x, size_t x_stride, size_t width, uint32_t tokens, uint32_t topk, const ExpertSource &src,
              const ExpertSink &sink, uint32_t align, uint32_t rows, void *out, size_t out_stride, cudaStream_t s)
{
    const uint32_t pieces = uint32_t(width / N), pads = uint32_t(gch::ceil_div(rows, kPadRows * (kRowThreads / 32)));
    const E *from = static_cast<const E *>(x);
    E *to = static_cast<E *>(out);
    if (tokens * topk <= kSmallPairs) {
        expert_small_kernel<E, N><<<tokens + pads, kRowThreads, 0, s>>>(src, sink, tokens * topk, topk, align, from,
                                                                        x_stride, rows, to, out_stride, pieces);
        return;
    }
    const dim3 block = row_block(pieces);
    const uint32_t spread = out ? uint32_t(gch::ceil_div(tokens, block.y)) : 0;
    gch::launch_next(expert_rows_kernel<E, N>, dim3(spread + pads), block, 0, s, from, x_stride, tokens, topk,
                     src.experts, static_cast<const int32_t *>(sink.offsets), static_cast<const int32_t *>(sink.counts),
                     static_cast<const int32_t *>(sink.slots), sink.pairs, rows, to, out_stride, pieces, spread);
}

// Row kernels by piece size: 16 bytes down to one element.
#define GC_BY_PIECE(T, n, CALL)                                     \
    switch (n) {                                                    \
    case 1: CALL(T, 1); break;                                      \
    case 2: CALL(T, 2); break;                                      \
    case 4: CALL(T, 4); break;                                      \
    default: CALL(T, (16 / int(sizeof(T)))); break;                 \
    }
#define GC_BY_DTYPE(dt, n, CALL)                                    \
    if (dt == GC_ROW_F32) { GC_BY_PIECE(float, n, CALL) }           \
    else if (dt == GC_ROW_BF16) { GC_BY_PIECE(__nv_bfloat16, n, CALL) } \
    else { GC_BY_PIECE(__half, n, CALL) }

}  // namespace

namespace gch {

size_t expert_workspace_bytes(size_t npairs, uint32_t experts)
{
    return npairs > kSmallPairs ? align_up(gcd::bin_table_bytes(npairs, experts), 256) + 256 : 256;
}

cudaError_t launch_expert_dispatch(const void *ids, bool wide, uint32_t npairs, uint32_t topk, uint32_t experts,
                                   uint32_t align, const void *x, size_t x_stride, size_t width, gc_row_dtype dt,
                                   void *out, size_t out_stride, uint32_t rows, int32_t *offsets, int32_t *counts,
                                   int32_t *slots, int32_t *pairs, uint8_t *ws, cudaStream_t s)
{
    uint32_t *table = reinterpret_cast<uint32_t *>(ws);
    const ExpertSource src{ids, wide, experts};
    const ExpertSink sink{offsets, counts, slots, pairs, experts};
    cudaError_t e = cudaSuccess;
    if (npairs > kSmallPairs) {
        e = gcd::launch_bin_count(src, npairs, experts, table, s);
        if (e == cudaSuccess) e = gcd::launch_bin_place(src, sink, npairs, experts, align, table, s);
    } else if (rows == 0) {  // no pairs either
        e = cudaMemsetAsync(offsets, 0, (size_t(experts) + 1) * sizeof(int32_t), s);
        if (e == cudaSuccess) e = cudaMemsetAsync(counts, 0, size_t(experts) * sizeof(int32_t), s);
        return e;
    }
    if (e != cudaSuccess) return e;
    const int elem = dt == GC_ROW_F32 ? 4 : 2;
    const int n = out ? piece_elems(uint64_t(uintptr_t(x)) | uintptr_t(out) | elem * (x_stride | out_stride | width), elem)
                      : 1;
#define GC_ROWS_CALL(E, N) run_rows<E, N>(x, x_stride, out ? width : 0, npairs / topk, topk, src, sink, align, rows, out, \
                                          out_stride, s)
    if (elem == 4) { GC_BY_PIECE(uint32_t, n, GC_ROWS_CALL) }
    else { GC_BY_PIECE(uint16_t, n, GC_ROWS_CALL) }
    return cudaGetLastError();
}

cudaError_t launch_expert_combine(const void *y, size_t y_stride, uint32_t rows, const int32_t *slots,
                                  const float *weights, uint32_t tokens, uint32_t topk, size_t width,
                                  gc_row_dtype dt, void *out, size_t out_stride, cudaStream_t s)
{
    const int elem = dt == GC_ROW_F32 ? 4 : 2;
    const int n = piece_elems(uint64_t(uintptr_t(y)) | uintptr_t(out) | elem * (y_stride | out_stride | width), elem);
#define GC_COMBINE_CALL(T, N) run_combine<T, N>(y, y_stride, rows, slots, weights, tokens, topk, width, out, out_stride, s)
    GC_BY_DTYPE(dt, n, GC_COMBINE_CALL)
    return cudaGetLastError();
}

cudaError_t launch_expert_combine_grad(const void *g, size_t g_stride, const void *y, size_t y_stride, uint32_t rows,
                                       const int32_t *slots, const int32_t *pairs, const float *weights,
                                       uint32_t tokens, uint32_t topk, size_t width, gc_row_dtype dt, void *dy,
                                       size_t dy_stride, float *dweights, cudaStream_t s)
{
    const int elem = dt == GC_ROW_F32 ? 4 : 2;
    uint64_t bits = uint64_t(uintptr_t(g)) | uintptr_t(dy) | elem * (g_stride | dy_stride | width);
    if (dweights) bits |= uintptr_t(y) | elem * y_stride;
    const int n = piece_elems(bits, elem);
#define GC_GRAD_CALL(T, N) run_combine_grad<T, N>(g, g_stride, y, y_stride, rows, slots, pairs, weights, tokens * topk, \
                                                  topk, width, dy, dy_stride, dweights, s)
    GC_BY_DTYPE(dt, n, GC_GRAD_CALL)
    return cudaGetLastError();
}

}  // namespace gch
