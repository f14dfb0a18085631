// cache.cu -- the scores of a cache's positions and the positions it keeps
// (gc_cache_score, gc_cache_evict).
//
// A score is the attention weight that a position has received: the old score
// times a decay, plus the sum over the queries and the heads that share the
// cache's head.  Eviction is a stable select-if whose predicate is "among the
// first or the last positions, or among the highest scores between them", with
// a row of keys and one of values attached to each element.
#include <atomic>

#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------- scores

constexpr int kScoreThreads = 256;
constexpr int kScoreRows = 8;   // rows that a thread has under way
constexpr uint32_t kScoreY = 8; // threads over the rows of one piece, at most

struct Weights {
    size_t batch_stride, head_stride, query_stride;
    uint32_t heads, group, queries, length;
    const int32_t *lengths, *counted;  // per sequence: positions, queries; NULL: all
};

__device__ __forceinline__ uint32_t clamp_length(const int32_t *lengths, uint32_t b, uint32_t most)
{
    return lengths ? uint32_t(min(max(lengths[b], 0), int32_t(most))) : most;
}

// Pieces across, the rows (queries of the group's heads, head by head) down the
// threads of a block, whose sums are then joined in their order.  Bound by HBM:
// 32 heads of 256 rows of 16384 bf16, 273 MB, take 46 us, 87% of the copy rate;
// with a row's address from two products and eight rows in local memory, as a
// tail of variable length left them, 98.  `whole`: the
// scores and the result move in 16 bytes too.
template <class T, int N>
__global__ void __launch_bounds__(kScoreThreads, 4)
cache_score_kernel(const T *__restrict__ weights, Weights a, const float *scores, size_t scores_stride, float decay,
                   float *out, size_t out_stride, uint32_t across, bool whole)
{
    __shared__ float s_acc[N][kScoreThreads];
    const uint32_t bh = blockIdx.x / across, b = bh / a.heads, h = bh % a.heads;
    const uint32_t first = (blockIdx.x % across * blockDim.x + threadIdx.x) * N;
    const uint32_t length = clamp_length(a.lengths, b, a.length), queries = clamp_length(a.counted, b, a.queries);
    float acc[N] = {};
    if (first < length && queries > 0) {
        const uint32_t rows = a.group * queries, y = blockDim.y;
        // from one of this thread's rows to the next: heads, and queries that may carry into one more
        const uint32_t dq = y % queries;
        const int64_t step = int64_t(y / queries) * int64_t(a.head_stride) + int64_t(dq) * int64_t(a.query_stride);
        const int64_t carry = int64_t(a.head_stride) - int64_t(queries) * int64_t(a.query_stride);
        uint32_t query = threadIdx.y % queries;
        const T *p = weights + size_t(b) * a.batch_stride +
                     (size_t(h) * a.group + threadIdx.y / queries) * a.head_stride + size_t(query) * a.query_stride +
                     first;
        auto next = [&] {
            p += step;
            query += dq;
            if (query >= queries) {
                query -= queries;
                p += carry;
            }
        };
        if (first + N <= a.length) {
            for (uint32_t r = threadIdx.y; r < rows; r += kScoreRows * y) {
                Piece<T, N> v[kScoreRows];
#pragma unroll
                for (int i = 0; i < kScoreRows; ++i) {
                    v[i] = r + i * y < rows ? load_piece<T, N>(p) : zero_piece<T, N>();
                    next();
                }
#pragma unroll
                for (int i = 0; i < kScoreRows; ++i) {
                    float x[N];
                    piece_values(v[i], x);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] += x[e];
                }
            }
        } else {  // the end of the rows
            for (uint32_t r = threadIdx.y; r < rows; r += y, next())
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (first + e < a.length) acc[e] += row_to_float(p[e]);
        }
    }
    if (blockDim.y > 1) {
        const uint32_t at = threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
        for (int e = 0; e < N; ++e) s_acc[e][at] = acc[e];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (uint32_t y = 1; y < blockDim.y; ++y)
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += s_acc[e][y * blockDim.x + threadIdx.x];
    }
    if (first >= a.length) return;
    const float *from = scores + size_t(bh) * scores_stride + first;
    float *to = out + size_t(bh) * out_stride + first;
    if (N >= 4 && whole && first + N <= a.length) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (scores && first + e < length) s = *reinterpret_cast<const float4 *>(from + e);
            float r[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float sum = acc[(e + k) % N];
                r[k] = first + e + k < length ? scores ? fmaf(decay, r[k], sum) : sum : 0.0f;
            }
            *reinterpret_cast<float4 *>(to + e) = make_float4(r[0], r[1], r[2], r[3]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (first + e >= a.length) break;
        to[e] = first + e < length ? scores ? fmaf(decay, from[e], acc[e]) : acc[e] : 0.0f;
    }
}

// ---------------------------------------------------------------- eviction

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr uint32_t kMaxTeam = 8;
constexpr int kBins = 4096;
static_assert(kBins == 4 * kEvictThreads && kEvictWarps == 32, "four bins to a thread, a lane to a warp");

struct Evict {
    uint32_t batch, heads, length, budget, sinks, recent;
    const float *scores;
    size_t scores_stride;
    const int32_t *positions;   // NULL: the index
    size_t positions_stride;
    const int32_t *lengths;     // NULL: all `length`
    float *kept_scores;
    int32_t *kept_positions, *kept_lengths;
    int32_t *list;              // workspace: [batch * heads][budget], the positions kept for their scores

    __host__ __device__ __forceinline__ uint32_t rows() const { return batch * heads; }
};

// Ascends with the score; NaN counts as -inf.
__device__ __forceinline__ uint32_t score_key(float x) { return order_bits(fmaxf(x, -INFINITY)); }

// Exclusive sum over the threads of a CTA.
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *s_warp)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, upto, o);
        if (lane >= uint32_t(o)) upto += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    return upto - v + __reduce_add_sync(kFull, lane < warp ? s_warp[lane] : 0u);
}

struct SelectSmem {
    alignas(16) uint32_t hist[kBins];
    uint32_t warp[kEvictWarps], equals[kEvictWarps];
    uint32_t bin, rest;
    uint32_t above, equal;  // this CTA's scores above the cut and at it
};

// The kept positions of one head of one sequence, by a cluster whose CTAs have
// a share of its positions each, and whose warps K * 32 neighbouring positions
// at a time, K to a lane, as ordered bits in registers.  The cut is the score of
// rank m between the sinks and the recent positions, found by three histograms
// of those bits, 12, 10 and 10 of them; of the scores at the cut the first are
// kept.  A share of at most K * 1024 positions is read once.  128 heads of 32768
// scores to 2048: 18 us, bound by instructions (62 of a warp for 32 scores, and 107
// with two CTAs to a head) between barriers, 52% of the issue slots; with four
// CTAs to a head that read their scores from L2 five times, 43.  All scores equal,
// each an atomic on one word three times: 22.
template <int K, int B>
__global__ void __launch_bounds__(kEvictThreads, B)
cache_select_kernel(Evict a)
{
    __shared__ SelectSmem sm;
    const uint32_t team = cluster_size(), rank = cluster_rank();
    const uint32_t bh = blockIdx.x / team, b = bh / a.heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t n = clamp_length(a.lengths, b, a.length), kept = min(n, a.budget);
    const float *scores = a.scores + size_t(bh) * a.scores_stride;
    int32_t *list = a.list + size_t(bh) * a.budget;
    chain_start();
    if (bh % a.heads == 0 && rank == 0 && threadIdx.x == 0) a.kept_lengths[b] = int32_t(kept);
    if (n <= a.budget) return;
    const uint32_t want = a.budget - a.sinks - a.recent;

    // this CTA's part of what lies between
    const uint32_t middle = n - a.recent - a.sinks;
    const uint32_t share = (middle + team - 1) / team;
    const uint32_t first = a.sinks + min(rank * share, middle), end = a.sinks + min((rank + 1) * share, middle);
    constexpr uint32_t kChunk = K * kEvictThreads;
    const bool once = end - first <= kChunk;
    uint32_t key[K];  // 0: no position
    extern __shared__ uint32_t s_turn[];
    // Read across the warp and turned in shared memory (rows of K + 1 words, so
    // that neither way meets a bank twice): K neighbouring positions to a lane.
    auto load = [&](uint32_t at) {
        uint32_t *mine = s_turn + warp * (32 * (K + 1));
        const uint32_t from = at + warp * (32 * K) + lane;
#pragma unroll
        for (int k = 0; k < K; ++k) key[k] = from + 32 * k < end ? score_key(scores[from + 32 * k]) : 0u;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t i = 32 * k + lane;
            mine[i / K * (K + 1) + i % K] = key[k];
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < K; ++k) key[k] = mine[lane * (K + 1) + k];
        __syncwarp();
    };
    if (want == 0) return;
    if (once) load(first);

    uint32_t cut = 0, rest = want;  // the cut's bits so far; the scores at or above the cut that are still to be found
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xfff00000u : 0xfffffc00u;
        const uint32_t bits = pass == 0 ? 4095u : 1023u;
        reinterpret_cast<uint4 *>(sm.hist)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (uint32_t at = first; at < end; at += kChunk) {
            if (!once) load(at);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (key[k] && (key[k] & mask) == cut) atomicAdd(&sm.hist[(key[k] >> shift) & bits], 1u);
        }
        cluster_sync();
        // from the highest bin down: thread i has bins kBins - 1 - 4 i and the three below
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        for (uint32_t q = 0; q < team; ++q) {
            const uint4 h = peer_load4(peer_address(sm.hist + kBins - 4 - 4 * threadIdx.x, q));
            c.x += h.w, c.y += h.z, c.z += h.y, c.w += h.x;
        }
        const uint32_t sum = c.x + c.y + c.z + c.w;
        uint32_t before = cta_scan(sum, sm.warp);
        if (before < rest && rest <= before + sum) {
            uint32_t k = 0;
            if (before + c.x < rest) {
                before += c.x, k = 1;
                if (before + c.y < rest) {
                    before += c.y, k = 2;
                    if (before + c.z < rest) before += c.z, k = 3;
                }
            }
            sm.bin = kBins - 1 - (4 * threadIdx.x + k);
            sm.rest = rest - before;
        }
        cluster_sync();  // the bin is known here, and nobody reads this histogram any more
        cut |= sm.bin << shift;
        rest = sm.rest;
    }

    // `rest` of the scores at the cut are kept: how many of either kind lie before this CTA's
    auto compare = [&](uint32_t &above, uint32_t &equal) {
        above = equal = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            above |= uint32_t(key[k] > cut) << k;
            equal |= uint32_t(key[k] == cut) << k;
        }
    };
    uint32_t up = 0, eq = 0, above, equal;
    if (team > 1) {
        uint32_t more = 0, same = 0;
        for (uint32_t at = first; at < end; at += kChunk) {
            if (!once) load(at);
            compare(above, equal);
            more += __popc(above), same += __popc(equal);
        }
        more = __reduce_add_sync(kFull, more);
        same = __reduce_add_sync(kFull, same);
        if (lane == 0) sm.warp[warp] = more, sm.equals[warp] = same;
        __syncthreads();
        if (warp == 0) {
            more = __reduce_add_sync(kFull, sm.warp[lane]);
            same = __reduce_add_sync(kFull, sm.equals[lane]);
            if (lane == 0) sm.above = more, sm.equal = same;
        }
        cluster_sync();
        for (uint32_t q = 0; q < rank; ++q) {
            up += peer_load(peer_address(&sm.above, q));
            eq += peer_load(peer_address(&sm.equal, q));
        }
        cluster_sync();  // nobody looks into another CTA any more
    }
    for (uint32_t at = first; at < end; at += kChunk) {
        if (!once) load(at);
        compare(above, equal);
        // of either kind before this lane's: in the low and the high half, in this warp at most K * 32
        const uint32_t mine = uint32_t(__popc(above)) | uint32_t(__popc(equal)) << 16;
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, upto, o);
            if (lane >= uint32_t(o)) upto += y;
        }
        __syncthreads();
        if (lane == 31) sm.warp[warp] = upto & 0xffffu, sm.equals[warp] = upto >> 16;
        __syncthreads();
        uint32_t my_up = up + __reduce_add_sync(kFull, lane < warp ? sm.warp[lane] : 0u) + ((upto - mine) & 0xffffu);
        uint32_t my_eq = eq + __reduce_add_sync(kFull, lane < warp ? sm.equals[lane] : 0u) + ((upto - mine) >> 16);
        up += __reduce_add_sync(kFull, sm.warp[lane]);
        eq += __reduce_add_sync(kFull, sm.equals[lane]);
        const uint32_t from = at + warp * (32 * K) + lane * K;
        for (uint32_t both = above | equal; both; both &= both - 1) {
            const uint32_t k = __ffs(both) - 1;
            const bool is_equal = equal >> k & 1u;
            if (!is_equal || my_eq < rest) {
                const uint32_t slot = a.sinks + my_up + min(my_eq, rest);
                if (slot < a.budget) list[slot] = int32_t(from + k);  // beyond it only if the scores change meanwhile
            }
            my_up += !is_equal;
            my_eq += is_equal;
        }
    }
}

struct RowArray {
    uint8_t *p;
    size_t batch, head, row;  // strides in bytes
};

struct Move {
    RowArray from[2], to[2];    // keys, values
    uint32_t pieces[2];         // of a row
    uint32_t piece[2];          // bytes of one: 2, 4, 8 or 16
    uint32_t across[2];         // threads to a row
    uint32_t arrays, slots;     // slots of a block
};

constexpr int kMoveThreads = 256;
constexpr int kMoveAhead = 4;   // rows that a thread has under way

// A block's slots of one array, each thread kMoveAhead rows at a time.
// position(slot) is a position, or `none`.
template <class P, class F>
__device__ __forceinline__ void move_rows(const uint8_t *from, size_t from_row, uint8_t *to, size_t to_row,
                                          uint32_t pieces, uint32_t across, uint32_t first, uint32_t end,
                                          uint32_t none, const F &position)
{
    const uint32_t down = kMoveThreads / across, x = threadIdx.x & (across - 1), y = threadIdx.x / across;
    for (uint32_t slot = first + y; slot < end; slot += kMoveAhead * down) {
        uint32_t at[kMoveAhead];
#pragma unroll
        for (int k = 0; k < kMoveAhead; ++k) at[k] = slot + k * down < end ? position(slot + k * down) : none;
        for (uint32_t c = x; c < pieces; c += across) {
            P v[kMoveAhead];
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k)
                if (at[k] < none) v[k] = reinterpret_cast<const P *>(from + size_t(at[k]) * from_row)[c];
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k)
                if (at[k] < none) reinterpret_cast<P *>(to + size_t(slot + k * down) * to_row)[c] = v[k];
        }
    }
}

// The kept rows, head by head; each array by the largest pieces that its own
// addresses allow.  Of `down` blocks of a head those that hold recent positions
// alone, the `early` last, come first for all heads: they need not wait for the
// selection.  128 heads of 2048 rows of 2 x 256 bytes: 44 us behind the
// selection's 18, for 268 MB (40 at the copy rate), each row a place of its own
// in HBM.  Blocks on an SM count for more than registers: with 4, 5, 6 and 8 of
// them 72, 67, 64 and 62 us altogether, though 8 spill 60 bytes; two rows at a
// time instead of four also 62, and 69 to 59 where rows have 66 bytes.
__global__ void __launch_bounds__(kMoveThreads, 8)
cache_move_kernel(Evict a, Move m, uint32_t down, uint32_t early)
{
    const uint32_t ahead = early * a.rows(), late = down - early;
    const bool is_early = blockIdx.x < ahead;
    const uint32_t unit = is_early ? blockIdx.x : blockIdx.x - ahead, each = is_early ? early : late;
    const uint32_t bh = unit / each, block = unit % each + (is_early ? late : 0);
    const uint32_t b = bh / a.heads, h = bh % a.heads, w = blockIdx.y;
    const uint32_t n = clamp_length(a.lengths, b, a.length), kept = min(n, a.budget);
    const uint32_t first = block * m.slots, end = min(first + m.slots, a.budget);
    // slots whose positions are known beforehand: those of the recent ones, of the sinks, and all of a short sequence
    const bool known = n <= a.budget || first >= a.budget - a.recent || end <= a.sinks;
    if (!known) chain_wait();
    const int32_t *list = a.list + size_t(bh) * a.budget;
    // the position of a slot, or a.length
    auto position = [&](uint32_t slot) {
        if (slot >= kept) return a.length;
        if (slot < a.sinks || n <= a.budget) return slot;
        if (slot >= a.budget - a.recent) return slot + (n - a.budget);
        return min(uint32_t(list[slot]), a.length);
    };
    if (w == m.arrays) {  // scores and positions, a thread to a slot
        const uint32_t slot = first + threadIdx.x;
        if (slot < end) {
            const uint32_t i = position(slot);
            float score = 0.0f;
            int32_t at = -1;
            if (i < a.length) {
                score = a.scores[size_t(bh) * a.scores_stride + i];
                at = a.positions ? a.positions[size_t(bh) * a.positions_stride + i] : int32_t(i);
            }
            a.kept_scores[size_t(bh) * a.budget + slot] = score;
            a.kept_positions[size_t(bh) * a.budget + slot] = at;
        }
    } else {
        const uint8_t *from = m.from[w].p + size_t(b) * m.from[w].batch + size_t(h) * m.from[w].head;
        uint8_t *to = m.to[w].p + size_t(b) * m.to[w].batch + size_t(h) * m.to[w].head;
        auto move = [&](auto piece) {
            move_rows<decltype(piece)>(from, m.from[w].row, to, m.to[w].row, m.pieces[w], m.across[w], first, end,
                                       a.length, position);
        };
        switch (m.piece[w]) {
        case 2: move(uint16_t()); break;
        case 4: move(uint32_t()); break;
        case 8: move(uint2()); break;
        default: move(uint4()); break;
        }
    }
    if (known) chain_wait();  // the launch is done when both kernels are
}

template <int K, int B>
cudaError_t run_select(cudaLaunchConfig_t cfg, const Evict &a)
{
    cfg.dynamicSmemBytes = kEvictWarps * 32 * (K + 1) * sizeof(uint32_t);
    // the attribute lasts as long as the process: set once for each device
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (e == cudaSuccess && (dev > 63 || !(set.load(std::memory_order_relaxed) & bit))) {
        e = cudaFuncSetAttribute(cache_select_kernel<K, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(cfg.dynamicSmemBytes));
        if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    }
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, cache_select_kernel<K, B>, a) : e;
}

template <class T, int N>
cudaError_t run_score(const void *weights, const Weights &a, uint32_t batch, const float *scores, size_t scores_stride,
                      float decay, float *out, size_t out_stride, cudaStream_t s)
{
    uint32_t y = 1;
    while (y < kScoreY && size_t(y) * kScoreRows < size_t(a.group) * a.queries) y <<= 1;
    const dim3 block(kScoreThreads / y, y);
    const uint32_t across = uint32_t(gch::ceil_div(a.length, size_t(block.x) * N));
    const bool whole = ((uintptr_t(scores) | uintptr_t(out) | 4 * (scores_stride | out_stride)) & 15u) == 0;
    cache_score_kernel<T, N><<<across * batch * a.heads, block, 0, s>>>(
        static_cast<const T *>(weights), a, scores, scores_stride, decay, out, out_stride, across, whole);
    return cudaGetLastError();
}

}  // namespace

namespace gch {

cudaError_t launch_cache_score(const void *weights, size_t batch_stride, size_t head_stride, size_t query_stride,
                               gc_row_dtype dt, uint32_t batch, uint32_t heads, uint32_t group, uint32_t queries,
                               uint32_t length, const float *scores, size_t scores_stride, float decay,
                               const int32_t *lengths, const int32_t *counted, float *out, size_t out_stride,
                               cudaStream_t s)
{
    const Weights a{batch_stride, head_stride, query_stride, heads, group, queries, length, lengths, counted};
    const int elem = dt == GC_ROW_F32 ? 4 : 2;
    const int n = piece_elems(uint64_t(uintptr_t(weights)) | elem * (batch_stride | head_stride | query_stride), elem);
#define GC_SCORE_CALL(T, N) return run_score<T, N>(weights, a, batch, scores, scores_stride, decay, out, out_stride, s)
#define GC_SCORE_BY_PIECE(T)                                  \
    switch (n) {                                              \
    case 1: GC_SCORE_CALL(T, 1);                              \
    case 2: GC_SCORE_CALL(T, 2);                              \
    case 4: GC_SCORE_CALL(T, 4);                              \
    default: GC_SCORE_CALL(T, (16 / int(sizeof(T))));         \
    }
    if (dt == GC_ROW_F32) { GC_SCORE_BY_PIECE(float) }
    if (dt == GC_ROW_BF16) { GC_SCORE_BY_PIECE(__nv_bfloat16) }
    GC_SCORE_BY_PIECE(__half)
}

size_t cache_evict_workspace_bytes(size_t rows, size_t budget) { return align_up(rows * budget * 4, 256) + 256; }

cudaError_t launch_cache_evict(const gc_cache_rows *keys, const gc_cache_rows *values, gc_row_dtype dt,
                               const float *scores, size_t scores_stride, const int32_t *positions,
                               size_t positions_stride, const int32_t *lengths, uint32_t batch, uint32_t heads,
                               uint32_t length, uint32_t budget, uint32_t sinks, uint32_t recent,
                               const gc_cache_rows *kept_keys, const gc_cache_rows *kept_values, float *kept_scores,
                               int32_t *kept_positions, int32_t *kept_lengths, uint8_t *ws, cudaStream_t s)
{
    const Evict a{batch, heads, length, budget, sinks, recent, scores, scores_stride, positions, positions_stride,
                  lengths, kept_scores, kept_positions, kept_lengths, reinterpret_cast<int32_t *>(ws)};
    const uint32_t rows = batch * heads;
    // A cluster per head: as many CTAs as read its positions once, 32 to a
    // thread, and up to four with 16 to a thread where all of them still run at a
    // time.  More meet too often: 8 heads of 32768 take 17 us by two CTAs each and
    // 25 by eight, of 131072 25 by four and 31 by eight.
    uint32_t team = 1;
    while (team < kMaxTeam && length > team * 32 * kEvictThreads) team *= 2;
    while (team < 4 && size_t(rows) * team * 2 <= kSms && length > team * 16 * kEvictThreads) team *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rows * team);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = team;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const uint32_t each = uint32_t(ceil_div(length, size_t(team) * kEvictThreads));
    // No more positions to a thread than the length needs (256 heads of 8000: 27 us
    // with 8, 42 with 32), and two CTAs to an SM, with half the registers, where
    // there are more than SMs (1024 heads of 5000: 65 us, 117 with 32 and one).
    const bool crowd = size_t(rows) * team > kSms;
    cudaError_t e;
    if (each <= 4) e = crowd ? run_select<4, 2>(cfg, a) : run_select<4, 1>(cfg, a);
    else if (each <= 8) e = crowd ? run_select<8, 2>(cfg, a) : run_select<8, 1>(cfg, a);
    else if (each <= 16) e = run_select<16, 1>(cfg, a);
    else e = run_select<32, 1>(cfg, a);
    if (e != cudaSuccess) return e;

    Move m{};
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const gc_cache_rows *from[2] = {keys, values}, *to[2] = {kept_keys, kept_values};
    m.arrays = values ? 2 : 1;
    for (uint32_t w = 0; w < m.arrays; ++w) {
        uint64_t bits = 0;
        auto put = [&](const gc_cache_rows &r) {
            const RowArray t{static_cast<uint8_t *>(r.d_rows), r.batch_stride * elem, r.head_stride * elem,
                             r.row_stride * elem};
            bits |= uint64_t(uintptr_t(t.p)) | t.batch | t.head | t.row | r.width * elem;
            return t;
        };
        m.from[w] = put(*from[w]);
        m.to[w] = put(*to[w]);
        m.piece[w] = uint32_t(piece_elems(bits, 2)) * 2;
        m.pieces[w] = uint32_t(from[w]->width * elem / m.piece[w]);
        for (m.across[w] = 1; m.across[w] < uint32_t(kMoveThreads) && m.across[w] < m.pieces[w];) m.across[w] *= 2;
    }
    // 64 slots to a block, fewer where that would leave SMs without one
    m.slots = 64;
    while (m.slots > 16 && size_t(rows) * ceil_div(budget, m.slots) < kSms * 4) m.slots /= 2;
    const uint32_t down = uint32_t(ceil_div(budget, m.slots)), early = down - uint32_t(ceil_div(budget - recent, m.slots));
    return launch_next(cache_move_kernel, dim3(down * rows, m.arrays + 1), dim3(kMoveThreads), 0, s, a, m, down, early);
}

}  // namespace gch
