// gc_binsort.cuh -- stable partition of n items into up to 2048 bins: the
// two-way partition's rank[i] with one counter per bin.
//
// The items are cut into at most kBinChunks contiguous chunks, one CTA each,
// and two kernels run: bin_count_kernel writes every chunk's count of every
// bin; bin_place_kernel adds the counts of the chunks before its own and of
// the smaller bins (each bin's total rounded up to `align`) to get where its
// first item of each bin goes, ranks its own items, and hands every item's
// destination to a sink.  Within a chunk a warp owns a contiguous segment and
// takes 32 items at a time, so the rank is: earlier warps' counts of the bin
// + this warp's count so far + the earlier lanes with the same bin.
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

// Exclusive scan of one value per thread over the CTA; total to every thread.
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
    for (int w = 0; w < kBinWarps; ++w) {
        const uint32_t c = s_warp[w];
        if (w < warp) before += c;
        total += c;
    }
    __syncthreads();
    return before + incl - v;
}

// Source: bin(i) in [0, bins], where `bins` marks an item that goes nowhere.
template <class Source>
__global__ void __launch_bounds__(kBinThreads)
bin_count_kernel(Source src, uint32_t n, uint32_t chunk, uint32_t bins, uint32_t *__restrict__ counts)
{
    __shared__ uint32_t s_hist[kMaxBins];
    for (uint32_t b = threadIdx.x; b < bins; b += kBinThreads) s_hist[b] = 0u;
    __syncthreads();
    const uint32_t first = blockIdx.x * chunk, last = min(n - first, chunk) + first;
    for (uint32_t i = first + threadIdx.x; i < last; i += kBinThreads) {
        const uint32_t b = src.bin(i);
        if (b < bins) atomicAdd(&s_hist[b], 1u);
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kBinThreads)
        counts[size_t(blockIdx.x) * bins + b] = s_hist[b];
}

// Sink: place(i, destination), drop(i); starts(b, start, count) once per bin
// and end(total) once, by CTA 0.  Dynamic shared memory: kBinWarps * bins
// words.
template <class Source, class Sink>
__global__ void __launch_bounds__(kBinThreads)
bin_place_kernel(Source src, Sink sink, uint32_t n, uint32_t chunk, uint32_t chunks, uint32_t bins,
                 uint32_t align, const uint32_t *__restrict__ counts)
{
    extern __shared__ uint32_t s_cnt[];  // [kBinWarps][bins]
    __shared__ uint32_t s_warp[kBinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (uint32_t i = tid; i < kBinWarps * bins; i += kBinThreads) s_cnt[i] = 0u;
    __syncthreads();

    const uint32_t first = blockIdx.x * chunk, size = n > first ? min(n - first, chunk) : 0u;
    const uint32_t segment = chunk / kBinWarps;  // a multiple of 32
    const uint32_t seg_lo = min(size, uint32_t(warp) * segment), seg_hi = min(size, seg_lo + segment);
    uint32_t *mine = s_cnt + size_t(warp) * bins;
    for (uint32_t i = seg_lo + lane; i < seg_hi; i += 32) {
        const uint32_t b = src.bin(first + i);
        if (b < bins) atomicAdd(&mine[b], 1u);
    }
    __syncthreads();

    // Per bin: items in earlier chunks and in all chunks; starts of the bins
    // by a scan over their rounded-up totals; then each warp's first
    // destination.
    const uint32_t per = (bins + kBinThreads - 1) / kBinThreads;
    const uint32_t lo = min(bins, uint32_t(tid) * per), hi = min(bins, lo + per);
    uint32_t sum = 0u;
    for (uint32_t b = lo; b < hi; ++b) {
        uint32_t all = 0u;
        for (uint32_t c = 0; c < chunks; ++c) all += counts[size_t(c) * bins + b];
        sum += (all + align - 1u) / align * align;
    }
    uint32_t total;
    uint32_t start = bin_block_scan(sum, s_warp, total);
    for (uint32_t b = lo; b < hi; ++b) {
        uint32_t all = 0u, before = 0u;
        for (uint32_t c = 0; c < chunks; ++c) {
            const uint32_t v = counts[size_t(c) * bins + b];
            if (c < blockIdx.x) before += v;
            all += v;
        }
        if (blockIdx.x == 0) sink.start(b, start, all);
        uint32_t at = start + before;
        for (int w = 0; w < kBinWarps; ++w) {
            const uint32_t v = s_cnt[size_t(w) * bins + b];
            s_cnt[size_t(w) * bins + b] = at;
            at += v;
        }
        start += (all + align - 1u) / align * align;
    }
    if (blockIdx.x == 0 && tid == 0) sink.end(total);
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

template <class Source>
cudaError_t launch_bin_count(const Source &src, uint32_t n, uint32_t bins, uint32_t *counts, cudaStream_t s)
{
    bin_count_kernel<Source><<<bin_chunks(n), kBinThreads, 0, s>>>(src, n, bin_chunk_elems(n), bins, counts);
    return cudaGetLastError();
}

template <class Source, class Sink>
cudaError_t launch_bin_place(const Source &src, const Sink &sink, uint32_t n, uint32_t bins,
                             uint32_t align, const uint32_t *counts, cudaStream_t s)
{
    auto kernel = bin_place_kernel<Source, Sink>;
    const size_t smem = size_t(kBinWarps) * bins * sizeof(uint32_t);
    const size_t most = size_t(kBinWarps) * kMaxBins * sizeof(uint32_t);
    // Raises the kernel's shared-memory limit, once per device.
    if (gch::persistent_grid(reinterpret_cast<const void *>(kernel), kBinThreads, most, 1) <= 0)
        return cudaErrorInvalidConfiguration;
    kernel<<<bin_chunks(n), kBinThreads, smem, s>>>(src, sink, n, bin_chunk_elems(n), bin_chunks(n), bins,
                                                   align, counts);
    return cudaGetLastError();
}

}  // namespace gcd
