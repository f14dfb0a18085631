// cache.cu -- the scores of a cache's positions and the positions it keeps
// (gc_cache_score, gc_cache_evict).
//
// A score is the attention weight that a position has received: the old score
// times a decay, plus the sum over the queries and the heads that share the
// cache's head.  Eviction is a stable select-if whose predicate is "among the
// first or the last positions, or among the highest scores between them", with
// a row of keys and one of values attached to each element.
#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------- scores

constexpr int kScoreRows = 8;   // rows that a thread has under way
constexpr int kScoreY = 8;      // threads over the rows of one piece, at most

struct Weights {
    size_t batch_stride, head_stride, query_stride;
    uint32_t heads, group, queries, length;
    const int32_t *lengths, *counted;  // per sequence: positions, queries; NULL: all
};

__device__ __forceinline__ uint32_t clamp_length(const int32_t *lengths, uint32_t b, uint32_t most)
{
    return lengths ? uint32_t(min(max(lengths[b], 0), int32_t(most))) : most;
}

// 32 pieces across, the rows (queries of the group's heads, head by head) down
// the threads of a block, then joined in their order.
template <class T, int N>
__global__ void __launch_bounds__(32 * kScoreY)
cache_score_kernel(const T *__restrict__ weights, Weights a, const float *scores, size_t scores_stride, float decay,
                   float *out, size_t out_stride, uint32_t across)
{
    __shared__ float s_acc[kScoreY][N][33];
    const uint32_t bh = blockIdx.x / across, b = bh / a.heads, h = bh % a.heads;
    const uint32_t first = (blockIdx.x % across * 32 + threadIdx.x) * N;
    const uint32_t length = clamp_length(a.lengths, b, a.length), queries = clamp_length(a.counted, b, a.queries);
    const T *base = weights + size_t(b) * a.batch_stride + size_t(h) * a.group * a.head_stride;
    float acc[N] = {};
    if (first < length && queries > 0) {
        const bool whole = first + N <= a.length;
        const uint32_t rows = a.group * queries;
        uint32_t head = threadIdx.y / queries, query = threadIdx.y % queries;
        for (uint32_t r = threadIdx.y; r < rows; r += kScoreRows * blockDim.y) {
            Piece<T, N> v[kScoreRows];
#pragma unroll
            for (int i = 0; i < kScoreRows; ++i) {
                v[i] = zero_piece<T, N>();
                if (r + i * blockDim.y < rows) {
                    const T *p = base + size_t(head) * a.head_stride + size_t(query) * a.query_stride + first;
                    if (whole) {
                        v[i] = load_piece<T, N>(p);
                    } else {
                        for (uint32_t e = 0; first + e < a.length; ++e) v[i].v[e] = p[e];
                    }
                }
                query += blockDim.y;
                while (query >= queries) query -= queries, ++head;
            }
#pragma unroll
            for (int i = 0; i < kScoreRows; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += row_to_float(v[i].v[e]);
        }
    }
    if (blockDim.y > 1) {
#pragma unroll
        for (int e = 0; e < N; ++e) s_acc[threadIdx.y][e][threadIdx.x] = acc[e];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (uint32_t y = 1; y < blockDim.y; ++y)
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += s_acc[y][e][threadIdx.x];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint32_t i = first + e;
        if (i >= a.length) break;
        float s = 0.0f;
        if (i < length) s = scores ? fmaf(decay, scores[size_t(bh) * scores_stride + i], acc[e]) : acc[e];
        out[size_t(bh) * out_stride + i] = s;
    }
}

// ---------------------------------------------------------------- eviction

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr uint32_t kMaxTeam = 8;
constexpr int kBins = 2048;
static_assert(kBins == 4 * kEvictThreads, "four bins to a thread");
constexpr uint32_t kTile = kEvictThreads * 4;

struct Evict {
    uint32_t batch, heads, length, budget, sinks, recent;
    const float *scores;
    size_t scores_stride;
    const int32_t *positions;   // NULL: the index
    size_t positions_stride;
    const int32_t *lengths;     // NULL: all `length`
    float *kept_scores;
    int32_t *kept_positions, *kept_lengths;
    int32_t *list;              // workspace: [batch * heads][budget] kept indices
};

// Ascends with the score; NaN is the least.
__device__ __forceinline__ uint32_t score_key(float x) { return order_bits(fmaxf(x, -INFINITY)); }

// Exclusive sum over the threads of a CTA; the total to all.
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t &total, uint32_t *s_warp)
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
    uint32_t w = lane < kEvictWarps ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < kEvictWarps; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, w, o);
        if (lane >= uint32_t(o)) w += y;
    }
    total = __shfl_sync(kFull, w, kEvictWarps - 1);
    const uint32_t before = __shfl_sync(kFull, w, warp ? warp - 1 : 0);
    return upto - v + (warp ? before : 0);
}

struct SelectSmem {
    alignas(16) uint32_t hist[kBins];
    uint32_t warp[kEvictWarps];
    uint32_t bin, rest;
    uint32_t above, equal;  // this CTA's scores above the cut and at it
};

// The kept positions of one head of one sequence, by a cluster.  The cut is the
// score of rank m between the sinks and the recent positions, found by three
// histograms of the ordered scores' bits, 11, 11 and 10 of them; of the scores
// at the cut the first are kept.
__global__ void __launch_bounds__(kEvictThreads)
cache_select_kernel(Evict a)
{
    __shared__ SelectSmem sm;
    const uint32_t team = cluster_size(), rank = cluster_rank();
    const uint32_t bh = blockIdx.x / team, b = bh / a.heads;
    const uint32_t n = clamp_length(a.lengths, b, a.length), kept = min(n, a.budget);
    const float *scores = a.scores + size_t(bh) * a.scores_stride;
    const int32_t *positions = a.positions ? a.positions + size_t(bh) * a.positions_stride : nullptr;
    int32_t *list = a.list + size_t(bh) * a.budget;
    float *to_scores = a.kept_scores + size_t(bh) * a.budget;
    int32_t *to_positions = a.kept_positions + size_t(bh) * a.budget;
    chain_start();
    auto keep = [&](uint32_t slot, uint32_t i, float x) {
        if (slot >= a.budget) return;  // only if the scores change meanwhile
        list[slot] = int32_t(i);
        to_scores[slot] = x;
        to_positions[slot] = positions ? positions[i] : int32_t(i);
    };
    const uint32_t me = rank * kEvictThreads + threadIdx.x, all = team * kEvictThreads;
    if (bh % a.heads == 0 && me == 0) a.kept_lengths[b] = int32_t(kept);
    for (uint32_t slot = kept + me; slot < a.budget; slot += all) {
        to_scores[slot] = 0.0f;
        to_positions[slot] = -1;
    }
    if (n <= a.budget) {
        for (uint32_t i = me; i < n; i += all) keep(i, i, scores[i]);
        return;
    }
    for (uint32_t i = me; i < a.sinks; i += all) keep(i, i, scores[i]);
    for (uint32_t i = me; i < a.recent; i += all)
        keep(a.budget - a.recent + i, n - a.recent + i, scores[n - a.recent + i]);
    const uint32_t want = a.budget - a.sinks - a.recent;
    if (want == 0) return;

    // this CTA's part of what lies between
    const uint32_t middle = n - a.recent - a.sinks;
    const uint32_t share = (middle + team - 1) / team;
    const uint32_t first = a.sinks + min(rank * share, middle), end = a.sinks + min((rank + 1) * share, middle);
    uint32_t cut = 0, rest = want;  // the cut's bits so far; the scores at or above the cut that are still to be found
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
        const uint32_t bits = pass == 2 ? 1023u : 2047u;
        reinterpret_cast<uint4 *>(sm.hist)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (uint32_t i = first + threadIdx.x; i < end; i += kEvictThreads) {
            const uint32_t key = score_key(scores[i]);
            if ((key & mask) == cut) atomicAdd(&sm.hist[(key >> shift) & bits], 1u);
        }
        cluster_sync();
        // from the highest bin down: thread i has bins kBins - 1 - 4 i and the three below
        uint32_t c[4] = {}, sum = 0;
        for (uint32_t q = 0; q < team; ++q) {
            const uint4 h = peer_load4(peer_address(sm.hist + kBins - 4 - 4 * threadIdx.x, q));
            c[0] += h.w, c[1] += h.z, c[2] += h.y, c[3] += h.x;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += c[k];
        uint32_t total, before = cta_scan(sum, total, sm.warp);
        if (before < rest && rest <= before + sum) {
            int k = 0;
            while (before + c[k] < rest) before += c[k++];
            sm.bin = kBins - 1 - (4 * threadIdx.x + k);
            sm.rest = rest - before;
        }
        cluster_sync();  // the bin is known here, and nobody reads this histogram any more
        cut |= sm.bin << shift;
        rest = sm.rest;
    }
    // `rest` of the scores at the cut are kept
    uint32_t above = 0, equal = 0;
    for (uint32_t i = first + threadIdx.x; i < end; i += kEvictThreads) {
        const uint32_t key = score_key(scores[i]);
        above += key > cut;
        equal += key == cut;
    }
    uint32_t total_above, total_equal;
    cta_scan(above, total_above, sm.warp);
    cta_scan(equal, total_equal, sm.warp);
    if (threadIdx.x == 0) sm.above = total_above, sm.equal = total_equal;
    cluster_sync();
    uint32_t above_before = 0, equal_before = 0;
    for (uint32_t q = 0; q < rank; ++q) {
        above_before += peer_load(peer_address(&sm.above, q));
        equal_before += peer_load(peer_address(&sm.equal, q));
    }
    cluster_sync();
    for (uint32_t base = first; base < end; base += kTile) {
        float x[4];
        uint32_t flags = 0, counts = 0;  // counts: above in the low half, equal in the high
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t i = base + 4 * threadIdx.x + k;
            if (i >= end) continue;
            x[k] = scores[i];
            const uint32_t key = score_key(x[k]);
            if (key > cut) flags |= 1u << k, counts += 1u;
            else if (key == cut) flags |= 16u << k, counts += 1u << 16;
        }
        uint32_t total, before = cta_scan(counts, total, sm.warp);
        uint32_t up = above_before + (before & 0xffffu), eq = equal_before + (before >> 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool is_above = flags >> k & 1u, is_equal = flags >> k & 16u;
            if (is_above || (is_equal && eq < rest)) keep(a.sinks + up + min(eq, rest), base + 4 * threadIdx.x + k, x[k]);
            up += is_above;
            eq += is_equal;
        }
        above_before += total & 0xffffu;
        equal_before += total >> 16;
    }
}

struct RowArray {
    uint8_t *p;
    size_t batch, head, row;  // strides in bytes
};

struct Move {
    RowArray from[2], to[2];    // keys, values
    uint32_t pieces[2];         // of sizeof(P) bytes
    uint32_t heads, length, budget;
    const int32_t *lengths, *list;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveAhead = 4;   // rows that a thread has under way

// The kept rows: a row of threads per slot, kMoveAhead slots at a time.
template <class P>
__global__ void __launch_bounds__(kMoveThreads)
cache_move_kernel(Move a, uint32_t down)
{
    chain_wait();
    const uint32_t bh = blockIdx.x / down, b = bh / a.heads, h = bh % a.heads, w = blockIdx.y;
    const uint32_t kept = min(clamp_length(a.lengths, b, a.length), a.budget);
    const uint32_t first = blockIdx.x % down * blockDim.y * kMoveAhead + threadIdx.y;
    if (first >= kept) return;
    const uint8_t *from = a.from[w].p + size_t(b) * a.from[w].batch + size_t(h) * a.from[w].head;
    uint8_t *to = a.to[w].p + size_t(b) * a.to[w].batch + size_t(h) * a.to[w].head;
    const int32_t *list = a.list + size_t(bh) * a.budget;
    uint32_t at[kMoveAhead];
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) {
        const uint32_t slot = first + k * blockDim.y;
        at[k] = slot < kept ? uint32_t(list[slot]) : ~0u;
    }
    for (uint32_t c = threadIdx.x; c < a.pieces[w]; c += blockDim.x) {
        P v[kMoveAhead];
#pragma unroll
        for (int k = 0; k < kMoveAhead; ++k)
            if (at[k] < a.length) v[k] = reinterpret_cast<const P *>(from + size_t(at[k]) * a.from[w].row)[c];
#pragma unroll
        for (int k = 0; k < kMoveAhead; ++k)
            if (at[k] < a.length)
                reinterpret_cast<P *>(to + size_t(first + k * blockDim.y) * a.to[w].row)[c] = v[k];
    }
}

template <class P>
cudaError_t run_move(Move a, uint32_t rows, uint32_t arrays, cudaStream_t s)
{
    uint32_t most = 1;
    for (uint32_t w = 0; w < arrays; ++w) {
        a.pieces[w] /= sizeof(P);
        most = a.pieces[w] > most ? a.pieces[w] : most;
    }
    uint32_t tx = 1;
    while (tx < kMoveThreads && tx < most) tx <<= 1;
    const dim3 block(tx, kMoveThreads / tx);
    const uint32_t down = uint32_t(gch::ceil_div(a.budget, block.y * kMoveAhead));
    return gch::launch_next(cache_move_kernel<P>, dim3(down * rows, arrays), block, 0, s, a, down);
}

template <class T, int N>
cudaError_t run_score(const void *weights, const Weights &a, uint32_t batch, const float *scores, size_t scores_stride,
                      float decay, float *out, size_t out_stride, cudaStream_t s)
{
    uint32_t y = 1;
    while (y < uint32_t(kScoreY) && size_t(y) * kScoreRows < size_t(a.group) * a.queries) y <<= 1;
    const uint32_t across = uint32_t(gch::ceil_div(a.length, 32 * N));
    cache_score_kernel<T, N><<<across * batch * a.heads, dim3(32, y), 0, s>>>(
        static_cast<const T *>(weights), a, scores, scores_stride, decay, out, out_stride, across);
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
    // A cluster per head: more CTAs where heads are few and caches long.
    uint32_t team = 1;
    while (team < kMaxTeam && size_t(rows) * team * 2 <= size_t(sm_count()) * 4 && length > team * kTile) team *= 2;
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, cache_select_kernel, a);
    if (e != cudaSuccess) return e;

    Move m{};
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const uint32_t arrays = values ? 2 : 1;
    uint64_t bits = 0;
    const gc_cache_rows *from[2] = {keys, values}, *to[2] = {kept_keys, kept_values};
    for (uint32_t w = 0; w < arrays; ++w) {
        auto put = [&](const gc_cache_rows &r) {
            const RowArray t{static_cast<uint8_t *>(r.d_rows), r.batch_stride * elem, r.head_stride * elem,
                             r.row_stride * elem};
            bits |= uint64_t(uintptr_t(t.p)) | t.batch | t.head | t.row | r.width * elem;
            return t;
        };
        m.from[w] = put(*from[w]);
        m.to[w] = put(*to[w]);
        m.pieces[w] = uint32_t(from[w]->width * elem);
    }
    m.heads = heads, m.length = length, m.budget = budget;
    m.lengths = lengths, m.list = a.list;
    switch (piece_elems(bits, 2) * 2) {
    case 2: return run_move<uint16_t>(m, rows, arrays, s);
    case 4: return run_move<uint32_t>(m, rows, arrays, s);
    case 8: return run_move<uint2>(m, rows, arrays, s);
    default: return run_move<uint4>(m, rows, arrays, s);
    }
}

}  // namespace gch
