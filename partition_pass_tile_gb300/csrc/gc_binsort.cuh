// gc_binsort.cuh -- stable partition of n items into up to 2048 bins: the
// two-way partition's rank[i] with one counter per bin.
//
// The items are cut into at most kBinChunks contiguous chunks, one CTA each,
// and two kernels run: bin_count_kernel writes every chunk's count of every
// bin; bin_place_kernel adds the counts of the chunks before its own and of
// the smaller bins (each bin's total rounded up to `align`) to get where its
// first item of each bin goes, ranks its own items, and hands every item's
// destination to a sink.  Within a chunk a warp owns a contiguous segment and
// takes 32 items at a time, so the rank is: earlier warps' counts of the bin +
// this warp's count so far + the earlier lanes with the same bin.  A single
// chunk needs no count kernel (bin_place_chunk with chunks == 1).  Both kernels
// are bound by latency: about 4 and 9 us for 32768 items in 512 bins, launch
// included; 256 threads or chunks of 512 or 2048 items are not faster.
#pragma once

#include "gc_internal.h"
#include "gc_rows.cuh"

namespace gcd {

constexpr int kBinThreads = 512;
constexpr int kBinWarps = kBinThreads / 32;
constexpr uint32_t kMaxBins = 2048;
constexpr uint32_t kBinChunks = 128;   // most chunks: every CTA reads all chunks' counts
constexpr uint32_t kBinMinChunk = 1024;

inline uint32_t bin_chunk_elems(size_t n)
{
    const size_t even = gch::align_up(gch::ceil_div(n, size_t(kBinChunks)), size_t(kBinThreads));
    return uint32_t(even > kBinMinChunk ? even : kBinMinChunk);
}
inline uint32_t bin_chunks(size_t n) { return uint32_t(gch::ceil_div(n, size_t(bin_chunk_elems(n)))); }
__host__ __device__ inline uint32_t bin_count_stride(uint32_t chunks) { return (chunks + 3u) / 4u * 4u; }
inline size_t bin_table_bytes(size_t n, size_t bins) { return size_t(bin_count_stride(bin_chunks(n))) * bins * 4; }

// Exclusive scan of one value per thread over THREADS threads; total to every
// thread.  Between two uses lies a barrier.
template <int THREADS>
__device__ __forceinline__ uint32_t bin_block_scan(uint32_t v, uint32_t *s_warp, uint32_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t before = 0u;
    total = 0u;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const uint32_t c = s_warp[w];
        if (w < warp) before += c;
        total += c;
    }
    return before + incl - v;
}

// Source: bin(i) in [0, bins], where `bins` marks an item that goes nowhere.
// Counts are written bin-major, counts[b * bin_count_stride(chunks) + c], with
// zeros up to the stride.
template <class Source>
__global__ void __launch_bounds__(kBinThreads)
bin_count_kernel(Source src, uint32_t n, uint32_t chunk, uint32_t bins,
                 uint32_t *__restrict__ counts)
{
    __shared__ uint32_t s_hist[kMaxBins];
    chain_start();
    chain_wait();
    for (uint32_t b = threadIdx.x; b < bins; b += kBinThreads) s_hist[b] = 0u;
    __syncthreads();
    const uint32_t first = blockIdx.x * chunk, last = min(n - first, chunk) + first;
    for (uint32_t i = first + threadIdx.x; i < last; i += kBinThreads) {
        const uint32_t b = src.bin(i);
        src.visit(i);
        if (b < bins) atomicAdd(&s_hist[b], 1u);
    }
    __syncthreads();
    const uint32_t chunks = gridDim.x, stride = bin_count_stride(chunks);
    for (uint32_t b = threadIdx.x; b < bins; b += kBinThreads) {
        counts[size_t(b) * stride + blockIdx.x] = s_hist[b];
        if (blockIdx.x == 0)
            for (uint32_t c = chunks; c < stride; ++c) counts[size_t(b) * stride + c] = 0u;
    }
}

struct BinSmem {
    uint32_t all[kMaxBins];     // items of each bin, then where the chunk's first goes
    uint32_t before[kMaxBins];  // of those, in earlier chunks
    uint32_t warp[kBinWarps];
};

// Places chunk `index` of `chunks` (bin_place_kernel); s_cnt: kBinWarps * bins
// words of shared memory.
template <class Source, class Sink>
__device__ __forceinline__ void bin_place_chunk(const Source &src, const Sink &sink, uint32_t n, uint32_t chunk,
                                                uint32_t chunks, uint32_t index, uint32_t bins, uint32_t align,
                                                const uint32_t *counts, uint32_t *s_cnt, BinSmem &sm)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (uint32_t i = tid; i < kBinWarps * bins; i += kBinThreads) s_cnt[i] = 0u;
    __syncthreads();

    const uint32_t first = index * chunk, size = n > first ? min(n - first, chunk) : 0u;
    const uint32_t segment = ((size + kBinThreads - 1) / kBinThreads) * 32u;  // per warp
    const uint32_t seg_lo = min(size, uint32_t(warp) * segment), seg_hi = min(size, seg_lo + segment);
    uint32_t *mine = s_cnt + size_t(warp) * bins;
    for (uint32_t i = seg_lo + lane; i < seg_hi; i += 32) {
        const uint32_t b = src.bin(first + i);
        if (chunks == 1) src.visit(first + i);
        if (b < bins) atomicAdd(&mine[b], 1u);
    }
    __syncthreads();

    // Per bin: items in all chunks and in earlier ones.  A group of lanes
    // reads one bin's counts, four chunks to a lane at a time.
    if (chunks == 1) {
        for (uint32_t b = tid; b < bins; b += kBinThreads) {
            uint32_t all = 0u;
#pragma unroll
            for (int w = 0; w < kBinWarps; ++w) all += s_cnt[size_t(w) * bins + b];
            sm.all[b] = all;
            sm.before[b] = 0u;
        }
    } else {
        uint32_t group = 1;
        while (group < 32 && bins * group * 2 <= kBinThreads) group <<= 1;
        const uint32_t quads = bin_count_stride(chunks) / 4, part = uint32_t(tid) & (group - 1);
        for (uint32_t base = 0; base < bins; base += kBinThreads / group) {  // the same for all lanes
            const uint32_t b = base + uint32_t(tid) / group;
            const uint4 *row = reinterpret_cast<const uint4 *>(counts) + size_t(b) * quads;
            uint32_t all = 0u, before = 0u;
            if (b < bins)
#pragma unroll 8
                for (uint32_t c = part; c < quads; c += group) {
                    const uint4 v = row[c];
                    all += v.x + v.y + v.z + v.w;
                    const uint32_t left = index > 4 * c ? index - 4 * c : 0u;  // chunks of the four before mine
                    before += (left > 0 ? v.x : 0u) + (left > 1 ? v.y : 0u) + (left > 2 ? v.z : 0u) +
                              (left > 3 ? v.w : 0u);
                }
            for (uint32_t o = 1; o < group; o <<= 1) {
                all += __shfl_xor_sync(0xffffffffu, all, o);
                before += __shfl_xor_sync(0xffffffffu, before, o);
            }
            if (b < bins && part == 0) {
                sm.all[b] = all;
                sm.before[b] = before;
            }
        }
    }
    __syncthreads();

    // Starts of the bins by a scan over their rounded-up totals, then each
    // warp's first destination.
    const uint32_t per = (bins + kBinThreads - 1) / kBinThreads;
    const uint32_t lo = min(bins, uint32_t(tid) * per), hi = min(bins, lo + per);
    uint32_t sum = 0u, total;
    for (uint32_t b = lo; b < hi; ++b) sum += (sm.all[b] + align - 1u) / align * align;
    uint32_t start = bin_block_scan<kBinThreads>(sum, sm.warp, total);
    for (uint32_t b = lo; b < hi; ++b) {
        const uint32_t all = sm.all[b];
        if (index == 0) sink.start(b, start, all);
        sm.all[b] = start + sm.before[b];
        start += (all + align - 1u) / align * align;
    }
    if (index == 0 && tid == 0) sink.end(total);
    __syncthreads();
    for (uint32_t b = tid; b < bins; b += kBinThreads) {
        uint32_t at = sm.all[b];
#pragma unroll
        for (int w = 0; w < kBinWarps; ++w) {
            const uint32_t v = s_cnt[size_t(w) * bins + b];
            s_cnt[size_t(w) * bins + b] = at;
            at += v;
        }
    }
    __syncthreads();

    for (uint32_t base = seg_lo; base < seg_hi; base += 32) {
        const uint32_t i = base + lane;
        const bool in = i < seg_hi;
        const uint32_t b = in ? src.bin(first + i) : bins;
        const uint32_t peers = __match_any_sync(0xffffffffu, b);
        const uint32_t lead = __ffs(peers) - 1;
        uint32_t at = 0u;
        if (b < bins && lane == int(lead)) {
            at = mine[b];
            mine[b] = at + __popc(peers);
        }
        __syncwarp();  // the next step's leader of this bin may be another lane
        at = __shfl_sync(0xffffffffu, at, lead) + __popc(peers & ((1u << lane) - 1u));
        if (in) {
            if (b < bins) sink.place(first + i, at);
            else sink.drop(first + i);
        }
    }
}

// Sink: place(i, destination), drop(i); start(b, start, count) once per bin
// and end(total) once, by CTA 0.  Dynamic shared memory: kBinWarps * bins
// words.
template <class Source, class Sink>
__global__ void __launch_bounds__(kBinThreads)
bin_place_kernel(Source src, Sink sink, uint32_t n, uint32_t chunk, uint32_t bins, uint32_t align,
                 const uint32_t *__restrict__ counts)
{
    extern __shared__ uint32_t s_cnt[];
    __shared__ BinSmem sm;
    chain_start();
    chain_wait();
    bin_place_chunk(src, sink, n, chunk, gridDim.x, blockIdx.x, bins, align, counts, s_cnt, sm);
}

// Both are kernels of a chain (launch_next), the count kernel its first
// unless `chained`.
template <class Source>
cudaError_t launch_bin_count(const Source &src, uint32_t n, uint32_t bins, uint32_t *counts, cudaStream_t s,
                             bool chained = false)
{
    auto kernel = bin_count_kernel<Source>;
    if (chained)
        return gch::launch_next(kernel, dim3(bin_chunks(n)), dim3(kBinThreads), 0, s, src, n, bin_chunk_elems(n), bins,
                                counts);
    kernel<<<bin_chunks(n), kBinThreads, 0, s>>>(src, n, bin_chunk_elems(n), bins, counts);
    return cudaGetLastError();
}

// Raises a kernel's shared-memory limit to what the most bins need, once per device.
inline bool bin_place_smem(const void *kernel)
{
    return gch::persistent_grid(kernel, kBinThreads, size_t(kBinWarps) * kMaxBins * sizeof(uint32_t), 1) > 0;
}

template <class Source, class Sink>
cudaError_t launch_bin_place(const Source &src, const Sink &sink, uint32_t n, uint32_t bins, uint32_t align,
                             const uint32_t *counts, cudaStream_t s)
{
    auto kernel = bin_place_kernel<Source, Sink>;
    if (!bin_place_smem(reinterpret_cast<const void *>(kernel))) return cudaErrorInvalidConfiguration;
    return gch::launch_next(kernel, dim3(bin_chunks(n)), dim3(kBinThreads),
                            size_t(kBinWarps) * bins * sizeof(uint32_t), s, src, sink, n, bin_chunk_elems(n), bins,
                            align, counts);
}

}  // namespace gcd
