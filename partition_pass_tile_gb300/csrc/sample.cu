// sample.cu -- one token per row of logits from given uniform random numbers
// (gc_sample): temperature, top-k, top-p, min-p, then the Gumbel-max draw.
//
// Every filter keeps a prefix of one order, x descending and equal values by
// index, which is the descending order of the 64-bit key
//     (order-preserving bits of x) << 32 | ~index,
// so a filter is a cut of that key.  Weights are added as whole multiples of
// 2^-40 of the largest weight wherever a sum decides a cut: such a sum does
// not depend on its order.
//
// A team of 1 to 8 CTAs (a cluster) owns a row; the first CTA is its leader.
//   - no cut (neither top-k nor top-p): one pass for the maximum, one for the
//     sum and the draw;
//   - a small top-k, or a short row: one pass collects the candidates, the
//     tokens not below a lower bound of the top_k-th largest value, in the
//     leader's shared memory, which sorts them and does the rest there;
//   - else each cut is found by a histogram of the tokens over z in steps of
//     1/64, a pass that collects the tokens around the cut's step and adds up
//     those above, and a sort of the collected; a last pass sums and draws.
//     Where the collected do not fit or do not hold the cut, the leader finds
//     it by radix selection over the whole row (select_cut).
#include <cooperative_groups.h>

#include "gc_internal.h"
#include "gc_rows.cuh"

namespace {

using namespace gcd;
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTeam = 8;
constexpr uint32_t kList = 4096;            // candidates that the leader can hold
constexpr int kBins = 2048;                 // histogram of z, 64 bins to a unit
constexpr float kBinsPerUnit = 64.0f;
constexpr int kLoads = 4;                   // 16-byte loads in flight per thread
constexpr float kFixed = 1099511627776.0f;  // 2^40
constexpr float kUniformLo = 0x1p-25f, kUniformHi = 1.0f - 0x1p-24f;

// x as the operator reads it: NaN is -inf, +inf the largest finite value.
__device__ __forceinline__ float sample_value(float x)
{
    return x != x ? -INFINITY : fminf(x, 3.402823466e38f);
}

// Ascends with x; -0 and +0 are one value.
__device__ __forceinline__ uint32_t order_bits(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    return (uint64_t(order_bits(x)) << 32) | uint32_t(~i);
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t o = uint32_t(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~uint32_t(key); }

__device__ __forceinline__ float scaled(float x, float m, float t)
{
    const float d = x - m;
    return d == -INFINITY ? d : d / t;
}

__device__ __forceinline__ uint64_t fixed_weight(float w) { return __float2ull_rn(w * kFixed); }

__device__ __forceinline__ float draw_score(float z, float u)
{
    return z - logf(-logf(fminf(fmaxf(u, kUniformLo), kUniformHi)));
}

struct Larger {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Plus {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};

struct Smem {
    uint64_t list[kList];
    uint32_t hist[kBins];
    uint64_t warp[kWarps];
    uint64_t slot[2][kMaxTeam];  // team reductions, two in turn
    uint64_t cut, above;
    uint32_t count;              // candidates appended (may pass kList)
    uint32_t bin;
    float threshold;
    bool found;
};

// A row as one thread of its team sees it: pieces of 16 bytes from the first
// aligned element on, and up to one piece's worth of single elements before
// and after them.
template <class T>
struct Row {
    static constexpr uint32_t kVec = 16 / sizeof(T);
    const T *x;
    uint32_t vocab, head, pieces, me, team;  // this thread and the threads of the team

    __device__ __forceinline__ Row(const T *x_, uint32_t vocab_, uint32_t rank, uint32_t size)
        : x(x_), vocab(vocab_), team(size * kThreads)
    {
        const uint32_t lead = uint32_t((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / uint32_t(sizeof(T));
        head = min(lead, vocab);
        pieces = (vocab - head) / kVec;
        me = rank * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ float value(uint32_t i) const { return sample_value(row_to_float(x[i])); }
    // Single elements outside the pieces; this thread's, or vocab.
    __device__ __forceinline__ uint32_t single() const
    {
        const uint32_t tail = head + pieces * kVec;
        if (me < head) return me;
        return me - head < vocab - tail ? tail + (me - head) : vocab;
    }
    // Piece q of the batch that starts at `base`, -inf past the end.
    __device__ __forceinline__ void load(uint32_t base, Piece<T, kVec> (&p)[kLoads]) const
    {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const uint32_t j = base + uint32_t(q) * team + me;
            if (j < pieces) {
                p[q] = load_piece<T, kVec>(x + head + size_t(j) * kVec);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) p[q].v[e] = row_from_float<T>(-INFINITY);
            }
        }
    }
    __device__ __forceinline__ uint32_t index(uint32_t base, int q, uint32_t e) const
    {
        return head + (base + uint32_t(q) * team + me) * kVec + e;
    }
    // f(value, index) for each of this thread's tokens that is not forbidden.
    template <class F>
    __device__ __forceinline__ void each(const F &f) const
    {
        const uint32_t s = single();
        if (s < vocab) {
            const float v = value(s);
            if (v > -INFINITY) f(v, s);
        }
        for (uint32_t base = 0; base < pieces; base += kLoads * team) {
            Piece<T, kVec> p[kLoads];
            load(base, p);
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) {
                    const float v = sample_value(row_to_float(p[q].v[e]));
                    if (v > -INFINITY) f(v, index(base, q, e));
                }
        }
    }
};

struct Team {
    Smem &sm;
    Smem *lead;  // the leader's shared memory
    uint32_t rank, size;
    int turn = 0;

    // The cluster, or this CTA alone.
    __device__ __forceinline__ Team(Smem &s, uint32_t size_) : sm(s), lead(&s), rank(0), size(size_)
    {
        if (size > 1) {
            rank = cg::this_cluster().block_rank();
            lead = peer(0);
        }
    }
    __device__ __forceinline__ Smem *peer(uint32_t c) const
    {
        return size > 1 ? cg::this_cluster().map_shared_rank(&sm, c) : &sm;
    }
    __device__ __forceinline__ void sync() const
    {
        if (size == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
    // The same value to every thread of the team.
    template <class Op>
    __device__ __forceinline__ uint64_t reduce(uint64_t v, Op op)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        __syncthreads();  // the previous use of sm.warp
        if ((threadIdx.x & 31) == 0) sm.warp[threadIdx.x >> 5] = v;
        __syncthreads();
        v = sm.warp[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = op(v, sm.warp[w]);
        if (size > 1) {
            // Slots alternate: a CTA writes a turn's slots again only two
            // reductions later, past a sync that follows every read.
            if (threadIdx.x < size) peer(threadIdx.x)->slot[turn][rank] = v;
            sync();
            v = sm.slot[turn][0];
            for (uint32_t c = 1; c < size; ++c) v = op(v, sm.slot[turn][c]);
            turn ^= 1;
        }
        return v;
    }
    // Adds this warp's keys to the leader's list; every lane calls it.
    __device__ __forceinline__ void append(bool mine, uint64_t key) const
    {
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (who == 0u) return;
        uint32_t at = 0u;
        const int first = __ffs(who) - 1, lane = threadIdx.x & 31;
        if (lane == first) at = atomicAdd(&lead->count, uint32_t(__popc(who)));
        at = __shfl_sync(0xffffffffu, at, first) + __popc(who & ((1u << lane) - 1u));
        if (mine && at < kList) lead->list[at] = key;
    }
};

// Exclusive scan over the CTA (u64), total to every thread.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, Smem &sm, uint64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) sm.warp[warp] = incl;
    __syncthreads();
    uint64_t before = 0u;
    total = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t c = sm.warp[w];
        if (w < warp) before += c;
        total += c;
    }
    return before + incl - v;
}

// Sorts list[0, n) descending (n <= kList; the list is padded with zeros,
// below every key), by the leader's CTA.
__device__ __forceinline__ void sort_list(Smem &sm, uint32_t n)
{
    uint32_t size = 2;
    while (size < n) size <<= 1;
    for (uint32_t i = n + threadIdx.x; i < size; i += kThreads) sm.list[i] = 0u;
    for (uint32_t run = 2; run <= size; run <<= 1)
        for (uint32_t step = run >> 1; step > 0; step >>= 1) {
            __syncthreads();
            for (uint32_t p = threadIdx.x; p < size / 2; p += kThreads) {
                const uint32_t i = 2 * p - (p & (step - 1)), j = i + step;
                const uint64_t a = sm.list[i], b = sm.list[j];
                if ((a < b) == ((i & run) == 0)) {
                    sm.list[i] = b;
                    sm.list[j] = a;
                }
            }
        }
    __syncthreads();
}

// The largest key K such that the amounts of all keys >= K sum to at least
// target (>= 1); 0 if they all together do not.  By radix selection, 8 bits a
// round, over the whole row by one CTA; its histogram is laid over the list.
// `each` calls its argument with every token's key and amount.
template <class Each>
__device__ __noinline__ uint64_t select_cut(uint64_t target, Smem &sm, const Each &each)
{
    uint64_t *hist = sm.list;
    uint64_t prefix = 0u, above = 0u;
    for (int shift = 56; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int b = threadIdx.x; b < 256; b += kThreads) hist[b] = 0u;
        if (threadIdx.x == 0) sm.found = false;
        __syncthreads();
        each([&](uint64_t key, uint64_t amount) {
            if (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(reinterpret_cast<unsigned long long *>(&hist[(key >> shift) & 255u]),
                          static_cast<unsigned long long>(amount));
        });
        __syncthreads();
        if (threadIdx.x < 32) {
            // Lane l owns bins 255 - 8 l down to 248 - 8 l.
            const int top = 255 - 8 * int(threadIdx.x);
            uint64_t sum = 0u;
            for (int k = 0; k < 8; ++k) sum += hist[top - k];
            uint64_t incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (int(threadIdx.x) >= o) incl += y;
            }
            uint64_t before = above + incl - sum;
            if (before < target && before + sum >= target) {
                for (int k = 0; k < 8; ++k) {
                    const uint64_t h = hist[top - k];
                    if (before < target && before + h >= target) {
                        sm.cut = prefix | (uint64_t(top - k) << shift);
                        sm.above = before;
                        sm.found = true;
                    }
                    before += h;
                }
            }
        }
        __syncthreads();
        if (!sm.found) return 0u;  // only in the first round: everything is kept
        prefix = sm.cut;
        above = sm.above;
    }
    return prefix;
}

// Bin of a token: its distance below the maximum in steps of 1/64; kBins for
// tokens 32 or more below, whose weights round to 0 of 2^-40.
__device__ __forceinline__ uint32_t z_bin(float z)
{
    const float b = -z * kBinsPerUnit;
    return b < float(kBins) ? uint32_t(b) : uint32_t(kBins);
}

// Amounts of a bin are counted in units of 2^shift, so that `bits` bits hold
// the largest weight of the bin and a bin of all tokens fits 32 bits.
__device__ __forceinline__ int bin_shift(uint32_t bin, int bits)
{
    const int top = 41 - int((bin * 1477u) >> 16);  // weights of the bin are below 2^top: 1477 / 2^16 < log2(e) / 64
    return max(0, top - bits);
}

// The cut at `target` (select_cut's) found by the team.  MASS: amounts are
// fixed-point weights and target is a share p of their sum; else each token
// counts 1 and target is k.  Only keys >= floor count.
template <bool MASS, class T>
__device__ __noinline__ uint64_t find_cut(Team &team, const Row<T> &row, float m, float t, uint64_t floor, uint64_t k,
                                          float p)
{
    Smem &sm = team.sm;
    const int bits = 32 - (32 - __clz(int(row.vocab)));
    team.sync();
    for (int b = threadIdx.x; b < kBins; b += kThreads) sm.hist[b] = 0u;
    if (threadIdx.x == 0) sm.count = 0u;
    team.sync();
    uint64_t total = 0u;
    row.each([&](float v, uint32_t i) {
        if (order_key(v, i) < floor) return;
        const float z = scaled(v, m, t);
        const uint32_t b = z_bin(z);
        if (b >= kBins) return;
        if (MASS) {
            const uint64_t w = fixed_weight(expf(z));
            const int s = bin_shift(b, bits);
            total += w;
            atomicAdd(&sm.hist[b], uint32_t((w + ((uint64_t(1) << s) >> 1)) >> s));
        } else {
            total += 1u;
            atomicAdd(&sm.hist[b], 1u);
        }
    });
    total = team.reduce(total, Plus());
    uint64_t target = k;
    if (MASS) {
        const double share = ceil(double(fmaxf(p, 0.0f)) * double(total));
        target = share < 1.0 ? 1u : uint64_t(share);
    } else if (total < k) {
        return 0u;  // the cut lies 32 below the maximum or more, where no weight is left
    }
    team.sync();  // every CTA's histogram is complete
    if (team.rank == 0) {
        // Thread j owns bins 4 j to 4 j + 3.
        constexpr int kPer = kBins / kThreads;
        uint64_t part[kPer], sum = 0u;
        for (int q = 0; q < kPer; ++q) {
            const uint32_t b = threadIdx.x * kPer + q;
            uint64_t h = 0u;
            for (uint32_t c = 0; c < team.size; ++c) h += team.peer(c)->hist[b];
            part[q] = MASS ? h << bin_shift(b, bits) : h;
            sum += part[q];
        }
        uint64_t all;
        uint64_t before = block_scan(sum, sm, all);
        const uint64_t aim = all < target ? all : target;  // rounding may leave the sum short
        if (before < aim && before + sum >= aim)
            for (int q = 0; q < kPer; ++q) {
                if (before < aim && before + part[q] >= aim) sm.bin = threadIdx.x * kPer + q;
                before += part[q];
            }
    }
    team.sync();
    // Tokens of the cut's bin and its neighbours to the list, those above added up.
    const uint32_t bin = team.lead->bin, lo = bin > 0 ? bin - 1 : 0;
    uint64_t above = 0u;
    {
        auto one = [&](float v, uint32_t i, bool in) {
            const uint64_t key = order_key(v, i);
            float z = 0.0f;
            uint32_t b = kBins;
            if (in && v > -INFINITY && key >= floor) {
                z = scaled(v, m, t);
                b = z_bin(z);
            }
            if (b < lo) above += MASS ? fixed_weight(expf(z)) : 1u;
            team.append(b >= lo && b <= bin + 1 && b < kBins, key);
        };
        const uint32_t s = row.single();
        one(s < row.vocab ? row.value(s) : -INFINITY, s, s < row.vocab);
        for (uint32_t base = 0; base < row.pieces; base += kLoads * row.team) {
            Piece<T, Row<T>::kVec> pc[kLoads];
            row.load(base, pc);
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
#pragma unroll
                for (uint32_t e = 0; e < Row<T>::kVec; ++e)
                    one(sample_value(row_to_float(pc[q].v[e])), row.index(base, q, e), true);
        }
    }
    above = team.reduce(above, Plus());
    team.sync();  // the list is complete
    if (team.rank == 0) {
        const uint32_t n = sm.count;
        if (threadIdx.x == 0) sm.found = false;
        if (n <= kList && above < target) {
            sort_list(sm, n);
            const uint32_t per = (n + kThreads - 1) / kThreads;
            const uint32_t first = min(n, threadIdx.x * per), last = min(n, first + per);
            auto amount = [&](uint32_t j) {
                return MASS ? fixed_weight(expf(scaled(key_value(sm.list[j]), m, t))) : uint64_t(1);
            };
            uint64_t sum = 0u, all;
            for (uint32_t j = first; j < last; ++j) sum += amount(j);
            uint64_t before = above + block_scan(sum, sm, all);
            for (uint32_t j = first; j < last; ++j) {
                const uint64_t a = amount(j);
                if (before < target && before + a >= target) {
                    sm.cut = sm.list[j];
                    sm.found = true;
                }
                before += a;
            }
        }
        __syncthreads();
        if (!sm.found) {
            const Row<T> whole(row.x, row.vocab, 0, 1);
            const uint64_t cut = select_cut(target, sm, [&](auto add) {
                whole.each([&](float v, uint32_t i) {
                    const uint64_t key = order_key(v, i);
                    if (key >= floor) add(key, MASS ? fixed_weight(expf(scaled(v, m, t))) : uint64_t(1));
                });
            });
            __syncthreads();
            if (threadIdx.x == 0) sm.cut = cut;
        }
    }
    team.sync();
    return team.lead->cut;
}

// The rest of a row whose candidates are all in the leader's list, by the
// leader's CTA: sort, top-k, top-p, min-p, draw.
__device__ __forceinline__ void finish_list(Smem &sm, uint32_t k, float t, float p, float q,
                                            const float *__restrict__ u, int32_t *token, float *logprob)
{
    const uint32_t n = min(k, sm.count);
    sort_list(sm, sm.count);
    const float m = key_value(sm.list[0]);
    const uint32_t per = (n + kThreads - 1) / kThreads;
    const uint32_t first = min(n, threadIdx.x * per), last = min(n, first + per);
    uint64_t before = 0u, target = ~uint64_t(0);
    if (p < 1.0f) {
        uint64_t sum = 0u, all;
        for (uint32_t j = first; j < last; ++j) sum += fixed_weight(expf(scaled(key_value(sm.list[j]), m, t)));
        before = block_scan(sum, sm, all);
        const double share = ceil(double(fmaxf(p, 0.0f)) * double(all));
        target = share < 1.0 ? 1u : uint64_t(share);
    }
    float sum = 0.0f;
    uint64_t best = 0u;
    for (uint32_t j = first; j < last && before < target; ++j) {
        const uint32_t i = key_index(sm.list[j]);
        const float z = scaled(key_value(sm.list[j]), m, t), w = expf(z);
        if (p < 1.0f) before += fixed_weight(w);
        if (w < q || w == 0.0f) continue;
        sum += w;
        if (z >= -20.0f) best = Larger()(best, order_key(draw_score(z, u[i]), i));
    }
    Team alone(sm, 1);
    best = alone.reduce(best, Larger());
    const uint64_t mass = alone.reduce(uint64_t(__double_as_longlong(double(sum))), [](uint64_t a, uint64_t b) {
        return uint64_t(__double_as_longlong(__longlong_as_double(int64_t(a)) + __longlong_as_double(int64_t(b))));
    });
    for (uint32_t j = threadIdx.x; j < n; j += kThreads)
        if (key_index(sm.list[j]) == key_index(best)) {
            *token = int32_t(key_index(best));
            if (logprob)
                *logprob = scaled(key_value(sm.list[j]), m, t) - logf(float(__longlong_as_double(int64_t(mass))));
        }
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const T *__restrict__ logits, size_t logits_stride, uint32_t vocab,
              const float *__restrict__ uniform, size_t uniform_stride, const float *__restrict__ temperature,
              const int32_t *__restrict__ top_k, const float *__restrict__ top_p, const float *__restrict__ min_p,
              int32_t *__restrict__ tokens, float *__restrict__ logprobs)
{
    __shared__ Smem sm;
    Team team(sm, cg::this_cluster().num_blocks());
    const uint32_t r = blockIdx.x / team.size;
    const Row<T> row(logits + size_t(r) * logits_stride, vocab, team.rank, team.size);
    const float *u = uniform + size_t(r) * uniform_stride;
    const float t = temperature ? temperature[r] : 1.0f;
    const float p = top_p ? top_p[r] : 1.0f;
    const float q0 = min_p ? min_p[r] : 0.0f, q = q0 > 0.0f ? fminf(q0, 1.0f) : 0.0f;
    const bool greedy = uniform == nullptr || !(t > 0.0f);
    const uint32_t k = top_k && top_k[r] > 0 ? min(uint32_t(top_k[r]), vocab) : vocab;
    int32_t *token = tokens + r;
    float *logprob = logprobs ? logprobs + r : nullptr;

    // Candidates by one pass: the whole row if it fits the list; else the
    // k-th largest of the threads' maxima over each CTA's first batch bounds
    // the k-th largest value from below, and about k in kBatch tokens get in.
    constexpr uint32_t kBatch = kLoads * kThreads * Row<T>::kVec;
    const bool shortcut = !greedy && (k < vocab || p < 1.0f) &&
                          (vocab <= kList || (k <= uint32_t(kThreads) && uint64_t(k) * vocab <= uint64_t(kBatch) * (kList * 3 / 4)));
    if (shortcut) {
        if (threadIdx.x == 0) {
            sm.count = 0u;
            sm.threshold = -INFINITY;
        }
        float threshold = -INFINITY;
        team.sync();
        Piece<T, Row<T>::kVec> pc[kLoads];
        row.load(0, pc);
        if (vocab > kList) {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < kLoads; ++b)
#pragma unroll
                for (uint32_t e = 0; e < Row<T>::kVec; ++e) top = fmaxf(top, sample_value(row_to_float(pc[b].v[e])));
            float *tops = reinterpret_cast<float *>(sm.hist);
            tops[threadIdx.x] = top;
            __syncthreads();
            uint32_t above = 0u;
            for (int j = 0; j < kThreads; j += 4) {
                const float4 o = *reinterpret_cast<const float4 *>(tops + j);
                above += (o.x > top || (o.x == top && j < int(threadIdx.x))) +
                         (o.y > top || (o.y == top && j + 1 < int(threadIdx.x))) +
                         (o.z > top || (o.z == top && j + 2 < int(threadIdx.x))) +
                         (o.w > top || (o.w == top && j + 3 < int(threadIdx.x)));
            }
            if (above == k - 1) sm.threshold = top;
            __syncthreads();
            threshold = sm.threshold;
        }
        const uint32_t s = row.single();
        const float sv = s < vocab ? row.value(s) : -INFINITY;
        team.append(sv > -INFINITY && sv >= threshold, order_key(sv, s));
        for (uint32_t base = 0; base < row.pieces;) {
#pragma unroll
            for (int b = 0; b < kLoads; ++b) {
                float top = -INFINITY;
#pragma unroll
                for (uint32_t e = 0; e < Row<T>::kVec; ++e) top = fmaxf(top, sample_value(row_to_float(pc[b].v[e])));
                if (!__any_sync(0xffffffffu, top > -INFINITY && top >= threshold)) continue;
#pragma unroll
                for (uint32_t e = 0; e < Row<T>::kVec; ++e) {
                    const float v = sample_value(row_to_float(pc[b].v[e]));
                    team.append(v > -INFINITY && v >= threshold, order_key(v, row.index(base, b, e)));
                }
            }
            base += kLoads * row.team;
            if (base < row.pieces) row.load(base, pc);
        }
        team.sync();
        const uint32_t n = team.lead->count;
        if (n <= kList) {
            if (team.rank == 0) {
                if (n > 0) {
                    finish_list(sm, k, t, p, q, u, token, logprob);
                } else if (threadIdx.x == 0) {
                    *token = -1;
                    if (logprob) *logprob = -INFINITY;
                }
            }
            team.sync();
            return;
        }
    }

    uint64_t best = 0u;
    row.each([&](float v, uint32_t i) { best = Larger()(best, order_key(v, i)); });
    best = team.reduce(best, Larger());
    if (best == 0u || greedy) {
        if (team.rank == 0 && threadIdx.x == 0) {
            *token = best == 0u ? -1 : int32_t(key_index(best));
            if (logprob) *logprob = best == 0u ? -INFINITY : 0.0f;
        }
        team.sync();
        return;
    }
    const float m = key_value(best);
    uint64_t cut = 0u;
    if (k < vocab) cut = find_cut<false>(team, row, m, t, 0u, k, 1.0f);
    if (p < 1.0f) cut = Larger()(cut, find_cut<true>(team, row, m, t, cut, 0u, p));

    // What is kept: its weight, and the draw.
    float sum = 0.0f;
    best = 0u;
    row.each([&](float v, uint32_t i) {
        if (order_key(v, i) < cut) return;
        const float z = scaled(v, m, t), w = expf(z);
        if (w < q || w == 0.0f) return;
        sum += w;
        if (z >= -20.0f) best = Larger()(best, order_key(draw_score(z, u[i]), i));
    });
    best = team.reduce(best, Larger());
    const uint64_t mass = team.reduce(uint64_t(__double_as_longlong(double(sum))), [](uint64_t a, uint64_t b) {
        return uint64_t(__double_as_longlong(__longlong_as_double(int64_t(a)) + __longlong_as_double(int64_t(b))));
    });
    if (team.rank == 0 && threadIdx.x == 0) {
        const uint32_t i = key_index(best);
        *token = int32_t(i);
        if (logprob) *logprob = scaled(row.value(i), m, t) - logf(float(__longlong_as_double(int64_t(mass))));
    }
    team.sync();  // no CTA leaves while another may read its shared memory
}

template <class T, class... A>
cudaError_t run_sample(const void *logits, uint32_t rows, uint32_t vocab, cudaStream_t s, size_t stride, A... args)
{
    // Few rows are spread over more SMs, down to one batch of a row per CTA.
    const uint64_t slots = 2u * uint64_t(gch::sm_count());
    uint32_t team = 1;
    while (team < kMaxTeam && uint64_t(rows) * (2 * team) <= slots &&
           vocab >= 2 * team * (kThreads * kLoads * uint32_t(16 / sizeof(T))))
        team *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rows * team);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = team;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, static_cast<const T *>(logits), stride, vocab, args...);
}

}  // namespace

namespace gch {

cudaError_t launch_sample(const void *logits, size_t logits_stride, uint32_t rows, uint32_t vocab, gc_row_dtype dt,
                          const float *uniform, size_t uniform_stride, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                          float *logprobs, cudaStream_t s)
{
    if (dt == GC_ROW_F32)
        return run_sample<float>(logits, rows, vocab, s, logits_stride, uniform, uniform_stride, temperature, top_k,
                                 top_p, min_p, tokens, logprobs);
    if (dt == GC_ROW_BF16)
        return run_sample<__nv_bfloat16>(logits, rows, vocab, s, logits_stride, uniform, uniform_stride, temperature,
                                         top_k, top_p, min_p, tokens, logprobs);
    return run_sample<__half>(logits, rows, vocab, s, logits_stride, uniform, uniform_stride, temperature, top_k,
                              top_p, min_p, tokens, logprobs);
}

}  // namespace gch
