// sample.cu -- one token per row of logits from given uniform random numbers
// (gc_sample): temperature, top-k, top-p, min-p, then the Gumbel-max draw.
//
// Every filter keeps a prefix of one order, x descending and equal values by
// index, which is the descending order of the 64-bit key
//     (order-preserving bits of x) << 32 | ~index,
// so a filter is a cut of that key.  Sums of weights are float32 trees whose
// order the row's length and the team's size decide, and, where atomics add or
// have decided the order (of a list), whole multiples of 2^-40 of the largest
// weight: the same call always finds the same cut, and gives the same bits.
//
// A team of 1 to 8 CTAs (a cluster) owns a row; the first CTA is its leader.
//   - no filter: one pass for the sum and the draw; min-p alone: one before it
//     for the maximum;
//   - a small top-k, or a short row: one pass collects the candidates, all
//     tokens or those not below a lower bound of the top_k-th largest value, and
//     the leader sorts a few of them and does the rest;
//   - else each cut is found by a histogram of the tokens over their weight, a
//     pass that collects the tokens about the cut's bin and adds up those
//     above, and a sort of few of the collected; the last cut's pass draws on
//     the way.  Where the collected do not fit (thousands of equal values) or do
//     not hold the cut, the leader finds it by radix selection (select_cut): 64
//     rows of 128000 equal bf16 logits take 0.6 ms, 100 us is usual.
// Measured, kernel alone, 512 x 128000 float32 (262 MB, 39 us at the copy rate)
// with nothing of it in L2: greedy 57 us; top-k 50 74 us against 295 by
// histograms; unfiltered 119 us (524 MB) in one pass against 199 in two; min-p
// 133 us, two passes; top-p 0.95 at T = 1.2 453 us, three reads of the logits,
// more than L2 holds, and most of the random numbers (1.10 GB); at T = 0.5 143
// us, one pass.  After a flush that leaves L2 dirty 4 to 10 us more.  One row of
// 128000 bf16: 13 us unfiltered or top-k, 44 us top-p.
// 512 threads at two CTAs per SM and rings of three pieces: more rows or pieces
// under way are slower (256 threads at four CTAs 109 us for top-k 50, rings of
// six 80, clusters of two 102), because HBM serves fewer, longer streams better.
#include <type_traits>

#include <cooperative_groups.h>

#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kResident = 2;                // CTAs per SM
constexpr uint32_t kMaxTeam = 8;
constexpr uint32_t kList = 4096;            // candidates that a CTA can hold
// Histogram of the distance below the maximum in powers of two, 64 bins to a
// power; from bin kBinsUsed on weights round to 0 of 2^-40.
constexpr int kBins = 4096;
constexpr uint32_t kBinsUsed = 42 * 64;
constexpr float kBinsPerPower = 64.0f;
constexpr int kSubBins = 1024;              // histogram of the list
constexpr uint32_t kFew = 1024;             // of the list's tokens near a cut
constexpr int kRing = 3;                    // pieces of 16 bytes that a thread has under way
constexpr int kSample = 8;                  // pieces per thread that bound the k-th largest value
constexpr float kFixed = 1099511627776.0f;  // 2^40
constexpr float kUniformLo = 0x1p-25f, kUniformHi = 1.0f - 0x1p-24f;
// -log u lies in [2^-24, 17.4] and the largest token weighs 1, so a token
// lighter than 2^-24 / 17.4 cannot be drawn; this is exp(-20).
constexpr float kLightest = 2.0611536e-9f;
constexpr uint32_t kFull = 0xffffffffu;

// x as the operator reads it: NaN is -inf, +inf the largest finite value.
__device__ __forceinline__ float sample_value(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f); }

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

__device__ __forceinline__ float order_value(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ float key_value(uint64_t key) { return order_value(uint32_t(key >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~uint32_t(key); }

// Tokens whose key is at least a cut, decided on the value: 0 keeps all.
struct Cut {
    float value;
    uint32_t index;
    __device__ __forceinline__ explicit Cut(uint64_t key)
        : value(key ? key_value(key) : -INFINITY), index(key ? key_index(key) : ~0u) {}
    __device__ __forceinline__ bool keeps(float x, uint32_t i) const { return x > value || (x == value && i <= index); }
};

// z = (x - m) / t and w = exp(z) of a row.  The quotient is a product with
// 1 / t, one rounding more and no division per token, and w a power of two,
// whose argument takes the same products.
struct Scale {
    float m, inv, power;  // power: log2(e) / t
    __device__ __forceinline__ Scale(float m_, float t) : m(m_)
    {
        inv = fminf(fmaxf(1.0f / t, 1.17549435e-38f), 3.402823466e38f);
        power = fminf(inv * 1.44269504f, 3.402823466e38f);
    }
    __device__ __forceinline__ float z(float x) const { return (x - m) * inv; }
    __device__ __forceinline__ float log_w(float x) const { return (x - m) * power; }  // to base 2
    __device__ __forceinline__ float w(float x) const { return exp2f(log_w(x)); }
    __device__ __forceinline__ uint64_t fixed(float x) const { return __float2ull_rn(w(x) * kFixed); }
};

// A sum of weights in units of 2^-40.
__device__ __forceinline__ float from_fixed(uint64_t units) { return __ull2float_rn(units) * (1.0f / kFixed); }

// The largest value of a piece; NaN counts for nothing.
template <class T, int N>
__device__ __forceinline__ float piece_max(const Piece<T, N> &p)
{
    if constexpr (sizeof(T) == 4) {
        float r = p.v[0];
#pragma unroll
        for (int e = 1; e < N; ++e) r = fmaxf(r, p.v[e]);
        return r;
    } else {
        // two at a time
        using Pair = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const Pair *q = reinterpret_cast<const Pair *>(p.v);
        Pair r = q[0];
#pragma unroll
        for (int e = 1; e < N / 2; ++e) r = __hmax2(r, q[e]);
        return fmaxf(row_to_float(T(r.x)), row_to_float(T(r.y)));
    }
}

// A key to find the largest of and a weight to add up, reduced together.
struct KeySum {
    uint64_t key;
    float sum;
};

struct Smem {
    uint4 ring[kRing][kThreads];
    uint64_t list[kList];        // candidates; the leader's, then all of them
    alignas(16) uint32_t hist[kBins];
    union {
        uint64_t sub[kSubBins];
        uint64_t few[kFew];
    };
    KeySum warp[2][kWarps];      // reductions, two in turn
    KeySum slot[2][kMaxTeam];
    uint64_t scan[kWarps];
    uint64_t cut, above;
    uint64_t units;              // kept weights of a list's tokens, in units of 2^-40 of the largest
    uint32_t count;              // candidates appended to this list (may pass kList)
    uint32_t bin, state;
    bool found;
};

// A row as one thread of its team sees it: pieces of 16 bytes from the first
// aligned element on, and up to one piece's worth of single elements before
// and after them.
template <class T>
struct Row {
    static constexpr uint32_t kVec = 16 / sizeof(T);
    const T *x;
    const float *u;
    uint32_t vocab, head, pieces, me, team;  // this thread and the threads of the team
    uint32_t shift;                          // elements of u between a 16-byte boundary and a piece's first

    __device__ __forceinline__ Row(const T *x_, const float *u_, uint32_t vocab_, uint32_t rank, uint32_t size)
        : x(x_), u(u_), vocab(vocab_), team(size * kThreads)
    {
        const uint32_t lead = uint32_t((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / uint32_t(sizeof(T));
        head = min(lead, vocab);
        pieces = (vocab - head) / kVec;
        me = rank * kThreads + threadIdx.x;
        shift = uint32_t(reinterpret_cast<uintptr_t>(u + head) >> 2) & 3u;
    }
    __device__ __forceinline__ float value(uint32_t i) const { return sample_value(row_to_float(x[i])); }
    // Single elements outside the pieces; this thread's, or vocab.
    __device__ __forceinline__ uint32_t single() const
    {
        const uint32_t tail = head + pieces * kVec;
        if (me < head) return me;
        return me - head < vocab - tail ? tail + (me - head) : vocab;
    }
    __device__ __forceinline__ void load(uint32_t j, Piece<T, kVec> &p) const
    {
        if (j < pieces) {
            p = load_piece<T, kVec>(x + head + size_t(j) * kVec);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) p.v[e] = row_from_float<T>(-INFINITY);
        }
    }
    // f(piece, its copy in shared memory, index of its first) for this thread's
    // pieces and, as a piece of one value, its single element; -inf where there
    // is no token.  All threads of a warp call f together.  The pieces come
    // through a ring of asynchronous copies, each thread's its own: kRing - 1 of
    // them are under way at any time, and f's code is there once, which matters
    // more than unrolling it (an unrolled f of the sizes below waits for
    // instructions).  With U the tokens' u come along, through a ring laid over
    // the list and the histogram, and f takes this thread's slot of it too: the
    // floats of a piece, four to a row of threads.
    template <bool U = false, class F>
    __device__ __forceinline__ void each(Smem &sm, const F &f) const
    {
        constexpr int kWords = kVec / 4;
        static_assert(sizeof(float4) * kRing * 2 * kThreads <= sizeof(sm.list) + sizeof(sm.hist), "ring of u");
        uint4 *ring = &sm.ring[0][threadIdx.x];
        float4 *uring = reinterpret_cast<float4 *>(sm.list) + threadIdx.x;
        Piece<T, kVec> none;
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) none.v[e] = row_from_float<T>(-INFINITY);
        auto copy = [&](uint32_t j, int slot) {
            if (j < pieces)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(
                                 __cvta_generic_to_shared(ring + slot * kThreads))),
                             "l"(x + head + size_t(j) * kVec)
                             : "memory");
            if (U && j < pieces) {
                const float *from = u + head + size_t(j) * kVec;
#pragma unroll
                for (int q = 0; q < kWords; ++q) {
                    const uint32_t to = uint32_t(__cvta_generic_to_shared(uring + (slot * kWords + q) * kThreads));
                    if (shift == 0) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from + 4 * q) : "memory");
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4u * e),
                                         "l"(from + 4 * q + e)
                                         : "memory");
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const uint32_t s = single();
        bool lone = __any_sync(kFull, s < vocab);
        if (!lone)
#pragma unroll
            for (int q = 0; q < kRing; ++q) copy(q * team + me, q);
        int slot = 0;
        for (uint32_t base = 0; lone || base < pieces;) {
            Piece<T, kVec> now = none;
            T *at = reinterpret_cast<T *>(ring + slot * kThreads);
            uint32_t i = s;
            if (lone) {
                if (s < vocab) now.v[0] = x[s];
                store_piece<T, kVec>(at, now);
                if (U) uring[0].x = s < vocab ? u[s] : 0.0f;
            } else {
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
                if (base + me < pieces) now = load_piece<T, kVec>(at);
                i = head + (base + me) * kVec;
            }
            if constexpr (U) f(now, static_cast<const T *>(at), i, static_cast<const float4 *>(uring + slot * kWords * kThreads));
            else f(now, static_cast<const T *>(at), i);
            if (lone) {
                lone = false;
#pragma unroll
                for (int q = 0; q < kRing; ++q) copy(q * team + me, q);
            } else {
                copy(base + kRing * team + me, slot);  // f is done with the slot
                slot = slot + 1 < kRing ? slot + 1 : 0;
                base += team;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    // u of the tokens of a piece, 0 past the end.
    __device__ __forceinline__ void uniforms(uint32_t i, float (&r)[kVec]) const
    {
        if (shift == 0 && i >= head && i + kVec <= vocab) {
#pragma unroll
            for (uint32_t e = 0; e < kVec; e += 4) {
                const float4 w = __ldcs(reinterpret_cast<const float4 *>(u + i + e));
                r[e] = w.x, r[e + 1] = w.y, r[e + 2] = w.z, r[e + 3] = w.w;
            }
        } else {
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) r[e] = i + e < vocab ? u[i + e] : 0.0f;
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
    // A CTA's shared memory may be touched by others only once it runs, which
    // no launch promises of a cluster's CTAs by itself: each announces itself
    // by started(), and nobody looks into another before all_started().  Both
    // together are a sync.
    __device__ __forceinline__ void started() const
    {
        if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    __device__ __forceinline__ void all_started() const
    {
        if (size == 1) __syncthreads();
        else asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // The same value to every thread of the team: the largest key and the sum,
    // added in a fixed order.  Buffers alternate: one is written again two
    // reductions later, past a barrier that follows every read of it.
    __device__ __noinline__ KeySum reduce(KeySum v)
    {
        auto join = [&](int o) {
            const uint64_t k = __shfl_xor_sync(kFull, v.key, o);
            v.key = k > v.key ? k : v.key;
            v.sum += __shfl_xor_sync(kFull, v.sum, o);
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) join(o);
        if ((threadIdx.x & 31) == 0) sm.warp[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = sm.warp[turn][threadIdx.x & (kWarps - 1)];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) join(o);
        if (size > 1) {
            if (threadIdx.x < size) peer(threadIdx.x)->slot[turn][rank] = v;
            sync();
            v = sm.slot[turn][threadIdx.x & (size - 1)];
            for (int o = int(size) / 2; o > 0; o >>= 1) join(o);
        }
        turn ^= 1;
        return v;
    }
    __device__ __forceinline__ uint64_t largest(uint64_t key) { return reduce(KeySum{key, 0.0f}).key; }
    __device__ __forceinline__ float sum(float v) { return reduce(KeySum{0u, v}).sum; }
    // Adds the tokens of a piece (in shared memory) with a bit in `which` to
    // this CTA's list.
    template <class T>
    __device__ __forceinline__ void append(uint32_t which, const T *x, uint32_t i) const
    {
        if (which == 0u) return;
        uint32_t at = atomicAdd(&sm.count, uint32_t(__popc(which)));
        for (; which; which &= which - 1, ++at) {
            const uint32_t e = __ffs(which) - 1;
            if (at < kList) sm.list[at] = order_key(sample_value(row_to_float(x[e])), i + e);
        }
    }
    // After a sync that follows every append: the tokens in all lists, to
    // every thread.  If they fit, the leader's list becomes all of them; its
    // threads read the others' lists as one.
    __device__ __forceinline__ uint32_t gather_lists() const
    {
        if (size == 1) return sm.count;
        const uint32_t lane = threadIdx.x & 31;
        uint32_t upto = lane < size ? peer(lane)->count : 0u;
#pragma unroll
        for (uint32_t o = 1; o < kMaxTeam; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t n = __shfl_sync(kFull, upto, size - 1), mine = __shfl_sync(kFull, upto, 0);
        if (rank == 0 && n <= kList)
            for (uint32_t base = mine; base < n; base += kThreads) {
                const uint32_t j = base + threadIdx.x;
                uint32_t c = 0u, start = 0u;
                for (uint32_t q = 0; q + 1 < size; ++q) {
                    const uint32_t end = __shfl_sync(kFull, upto, q);
                    if (j >= end) {
                        c = q + 1;
                        start = end;
                    }
                }
                if (j < n) sm.list[j] = peer(c)->list[j - start];
            }
        __syncthreads();
        return n;
    }
};

// The draw: of the tokens offered, the largest w / -log u, which orders them
// as z - log(-log u) does.  A token can only be it if -log u < w / bound for
// any ratio `bound` already seen, so u > 1 - w / bound: one multiply-add
// spares most tokens the logarithm.
struct Draw {
    float best = -1.0f;
    uint32_t index = ~0u;
    float bound = 0.0f, slope = -INFINITY;  // bound: the warp's; slope: -1 / bound and a little more

    __device__ __forceinline__ bool open(float w, float u) const { return u >= fmaf(w, slope, 0.9999995f); }
    __device__ __forceinline__ void take(float w, float u, uint32_t i)
    {
        const float r = w / -logf(fminf(fmaxf(u, kUniformLo), kUniformHi));
        if (r > best || (r == best && i < index)) {
            best = r;
            index = i;
        }
    }
    // All lanes together: the bound of the warp.
    __device__ __forceinline__ void share()
    {
        float b = best;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) b = fmaxf(b, __shfl_xor_sync(kFull, b, o));
        if (b > bound) {
            bound = b;
            slope = -1.00001f / b;
        }
    }
    // Offers the tokens of a piece with a bit in `kept`; all lanes together.
    template <uint32_t N, class T>
    __device__ __forceinline__ void offer(const float (&w)[N], uint32_t kept, const float (&u)[N], const Row<T> &row,
                                          const Scale &scale, const T *x, uint32_t i)
    {
        uint32_t any = 0u;
#pragma unroll
        for (uint32_t e = 0; e < N; ++e) any |= open(w[e], fmaxf(u[e], kUniformLo)) ? 1u << e : 0u;
        any &= kept;
        if (!__any_sync(kFull, any != 0u)) return;
        for (; any; any &= any - 1) {
            const uint32_t e = __ffs(any) - 1;
            take(scale.w(sample_value(row_to_float(x[e]))), row.u[i + e], i + e);
        }
        __syncwarp();
        share();
    }
    __device__ __forceinline__ uint64_t key() const { return best > 0.0f ? order_key(best, index) : 0u; }
};

// Exclusive scan over the CTA (u64), total to every thread.  Between two uses
// lies a barrier.
__device__ __noinline__ uint64_t block_scan(uint64_t v, Smem &sm, uint64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    uint64_t c = lane < kWarps ? sm.scan[lane] : 0u;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, c, o);
        if (lane >= o) c += y;
    }
    total = __shfl_sync(kFull, c, kWarps - 1);
    const uint64_t before = __shfl_sync(kFull, c, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0u) + incl - v;
}

// Adds v to *sum (in shared memory), by all lanes of the warp together; a
// barrier lies between the last and who reads it.
__device__ __forceinline__ void add_units(uint64_t v, uint64_t *sum)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0 && v != 0u)
        atomicAdd(reinterpret_cast<unsigned long long *>(sum), static_cast<unsigned long long>(v));
}

// Sorts up to 64 keys descending, two to a lane of one warp.
__device__ __forceinline__ void sort_warp(uint64_t *list, uint32_t n)
{
    const uint32_t lane = threadIdx.x & 31;
    uint64_t a = lane < n ? list[lane] : 0u, b = lane + 32 < n ? list[lane + 32] : 0u;
#pragma unroll
    for (uint32_t run = 2; run <= 64; run <<= 1) {
        if (run == 64) {
            const uint64_t hi = a > b ? a : b;
            b = a > b ? b : a;
            a = hi;
        }
#pragma unroll
        for (uint32_t step = run >> 1 > 16 ? 16 : run >> 1; step > 0; step >>= 1) {
            const uint64_t x = __shfl_xor_sync(kFull, a, step), y = __shfl_xor_sync(kFull, b, step);
            const bool low = (lane & step) == 0;
            // Key i = lane (a) or lane + 32 (b) goes down in runs with i & run == 0.
            a = (a > x) == (low == ((lane & run) == 0)) ? a : x;
            b = (b > y) == (low == (((lane + 32) & run) == 0)) ? b : y;
        }
    }
    if (lane < n) list[lane] = a;
    if (lane + 32 < n) list[lane + 32] = b;
}

// Sorts list[0, n) descending, by one CTA; the list has room for the next
// power of two and is padded with zeros, below every key.
__device__ __noinline__ void sort_list(uint64_t *list, uint32_t n)
{
    __syncthreads();
    if (n <= 64) {
        if (threadIdx.x < 32) sort_warp(list, n);
    } else {
        uint32_t size = 128;
        while (size < n) size <<= 1;
        for (uint32_t i = n + threadIdx.x; i < size; i += kThreads) list[i] = 0u;
        for (uint32_t run = 2; run <= size; run <<= 1)
            for (uint32_t step = run >> 1; step > 0; step >>= 1) {
                __syncthreads();
                for (uint32_t p = threadIdx.x; p < size / 2; p += kThreads) {
                    const uint32_t i = 2 * p - (p & (step - 1)), j = i + step;
                    const uint64_t a = list[i], b = list[j];
                    if ((a < b) == ((i & run) == 0)) {
                        list[i] = b;
                        list[j] = a;
                    }
                }
            }
    }
    __syncthreads();
}

// Where of the list a cut falls, by one CTA: the bin of a histogram over
// (top - x) * rate, and the amounts of the bins before it and of the tokens
// `before` the list; kSubBins where the list does not reach the target.  With
// `open` the last bin is not counted: it is where thousands of tokens without
// weight may lie, whose atomics would follow one another (400 rows of 4000, top-k
// with top-p: 123 us so, 18 without).
struct SubBin {
    float top, rate;
    uint32_t at;
    uint64_t before;
    __device__ __forceinline__ uint32_t of(uint64_t key) const
    {
        return uint32_t(fminf(fmaxf((top - key_value(key)) * rate, 0.0f), float(kSubBins - 1)));
    }
};

template <class Amount>
__device__ __forceinline__ SubBin sub_bin(Smem &sm, uint32_t n, float top, float span, bool open, uint64_t before,
                                          uint64_t target, const Amount &amount)
{
    SubBin r{top, float(kSubBins) / fmaxf(span, 1e-30f), kSubBins, 0u};
    __syncthreads();
    for (int b = threadIdx.x; b < kSubBins; b += kThreads) sm.sub[b] = 0u;
    if (threadIdx.x == 0) sm.bin = kSubBins;
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < n; j += kThreads) {
        const uint32_t b = r.of(sm.list[j]);
        if (!open || b + 1 < uint32_t(kSubBins))
            atomicAdd(reinterpret_cast<unsigned long long *>(&sm.sub[b]),
                      static_cast<unsigned long long>(amount(sm.list[j])));
    }
    __syncthreads();
    constexpr int kPer = kSubBins / kThreads;
    uint64_t part[kPer], sum = 0u, all;
#pragma unroll
    for (int q = 0; q < kPer; ++q) sum += part[q] = sm.sub[threadIdx.x * kPer + q];
    uint64_t at = before + block_scan(sum, sm, all);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        if (at < target && at + part[q] >= target) {
            sm.bin = threadIdx.x * kPer + q;
            sm.above = at;
        }
        at += part[q];
    }
    __syncthreads();
    r.at = sm.bin;
    r.before = sm.above;
    return r;
}

// The list's keys with pick(key) to sm.few; how many there are (may pass kFew).
template <class Pick>
__device__ __forceinline__ uint32_t pick_few(Smem &sm, uint32_t n, const Pick &pick)
{
    __syncthreads();
    if (threadIdx.x == 0) sm.count = 0u;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (uint32_t base = 0; base < n; base += kThreads) {
        const uint32_t j = base + threadIdx.x;
        const uint64_t key = j < n ? sm.list[j] : 0u;
        const bool mine = j < n && pick(key);
        const uint32_t who = __ballot_sync(kFull, mine);
        if (who == 0u) continue;
        uint32_t at = 0u;
        const int first = __ffs(who) - 1;
        if (lane == first) at = atomicAdd(&sm.count, uint32_t(__popc(who)));
        at = __shfl_sync(kFull, at, first) + __popc(who & ((1u << lane) - 1u));
        if (mine && at < kFew) sm.few[at] = key;
    }
    __syncthreads();
    return sm.count;
}

// The largest K of 16 leading bits such that at least k of the CTA's order
// bits, one per thread, are >= K, the bits below them 0; 0 if there are fewer.
__device__ __forceinline__ uint32_t kth_largest(uint32_t o, uint32_t k)
{
    uint32_t at = 0u;
#pragma unroll 1
    for (int b = 31; b >= 16; --b) {
        const uint32_t mid = at | (1u << b);
        if (uint32_t(__syncthreads_count(o >= mid)) >= k) at = mid;
    }
    return at;
}

// The largest key K such that `above` and the amounts of all keys >= K sum to
// at least target (> above); 0 if they all together do not.  By radix
// selection, 8 bits a round, over the whole row by one CTA; its histogram is
// laid over the list.  `each` calls its argument with the tokens' keys and
// amounts.
template <class Each>
__device__ __noinline__ uint64_t select_cut(uint64_t target, uint64_t above, Smem &sm, const Each &each)
{
    uint64_t *hist = sm.list;
    uint64_t prefix = 0u;
    for (int shift = 56; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int b = threadIdx.x; b < 256; b += kThreads) hist[b] = 0u;
        if (threadIdx.x == 0) sm.found = false;
        __syncthreads();
        // Equal values, of which there are many where this is needed, fall in
        // one bin: a thread adds up what follows in the same bin.
        uint32_t bin = 0u;
        uint64_t sum = 0u;
        auto flush = [&]() {
            if (sum)
                atomicAdd(reinterpret_cast<unsigned long long *>(&hist[bin]), static_cast<unsigned long long>(sum));
        };
        each([&](uint64_t key, uint64_t amount) {
            if (shift != 56 && (key >> (shift + 8)) != (prefix >> (shift + 8))) return;
            const uint32_t b = uint32_t(key >> shift) & 255u;
            if (b != bin) {
                flush();
                bin = b;
                sum = 0u;
            }
            sum += amount;
        });
        flush();
        __syncthreads();
        if (threadIdx.x < 32) {
            // Lane l owns bins 255 - 8 l down to 248 - 8 l.
            const int top = 255 - 8 * int(threadIdx.x);
            uint64_t sum = 0u;
            for (int k = 0; k < 8; ++k) sum += hist[top - k];
            uint64_t incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(kFull, incl, o);
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
        if (!sm.found) return 0u;  // only in the first round: all of them do not reach it
        prefix = sm.cut;
        above = sm.above;
    }
    return prefix;
}

// x rounded to a whole number, 0 <= x < 2^22: an addition that leaves it in the
// low bits; a conversion instruction takes eight times its issue slots.
__device__ __forceinline__ uint32_t round_small(float x) { return __float_as_uint(x + 8388608.0f) & 0x7fffffu; }

// Bin of a token from the base-2 logarithm of its weight, rounded; kBinsUsed
// and more: no weight, or NaN.
__device__ __forceinline__ uint32_t weight_bin(float log_w)
{
    return round_small(fminf(log_w * -kBinsPerPower, float(kBins - 1)));
}

// A bin's weights, all below 2^(1 - e) for e = its power, are counted in units
// of 2^-(e + bits), 2^bits times the vocabulary at most 2^31, so that a bin of
// all tokens fits 32 bits.
__device__ __forceinline__ int bin_power(uint32_t bin) { return int(bin >> 6); }

__device__ __forceinline__ uint64_t share_of(float p, double fixed_sum)
{
    const double s = ceil(double(fmaxf(p, 0.0f)) * fixed_sum);
    return s < 1.0 ? 1u : uint64_t(s);
}

// Whether find_cut found the cut, may find it with other bins, or cannot.
enum : uint32_t { kMissed, kFound, kAgain };

// What the row keeps so far: the sum of the weights and the draw.
struct Kept {
    float sum = 0.0f;
    Draw draw;
};

// The cut at `target` (select_cut's) found by the team.  MASS: amounts are
// weights and the target is a share p of their sum; else each token counts 1
// and the target is k.  FLOOR: only the tokens of `floor` count.  With `kept`,
// the tokens above the cut's bins are added to it on the way and the leader
// adds the rest; returns whether it did.
template <bool MASS, bool FLOOR, class T>
__device__ __noinline__ bool find_cut(Team &team, const Row<T> &row, const Scale &row_scale, uint64_t floor_key,
                                      uint32_t k, float p, float q, Kept *kept, uint64_t &cut_key)
{
    constexpr uint32_t kVec = Row<T>::kVec;
    Smem &sm = team.sm;
    const Scale scale = row_scale;
    const Cut floor(floor_key);
    const int bits = min(14, __clz(int(row.vocab)) - 1);
    for (int b = threadIdx.x; b < kBins; b += kThreads) sm.hist[b] = 0u;
    team.sync();
    float mass = 0.0f;
    row.each(sm, [&](const Piece<T, kVec> &x, const T *, uint32_t i) {
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) {
            const float v = sample_value(row_to_float(x.v[e])), l = scale.log_w(v);
            const uint32_t b = weight_bin(l);
            if (b >= kBinsUsed || (FLOOR && !floor.keeps(v, i + e))) continue;
            if (MASS) {
                const float w = exp2f(l);
                mass += w;
                atomicAdd(&sm.hist[b], round_small(w * __int_as_float((127 + bits + bin_power(b)) << 23)));
            } else {
                mass += 1.0f;
                atomicAdd(&sm.hist[b], 1u);
            }
        }
    });
    mass = team.sum(mass);
    uint64_t target = k;
    if (MASS) {
        target = share_of(p, double(mass) * double(kFixed));
    } else if (mass < float(k)) {
        cut_key = floor_key;  // the cut lies where no weight is left
        return false;
    }
    // The rounded amounts may miss the cut's bin where the bins about it hold
    // next to nothing; the exact sum above the bins tried puts that right.
    int64_t error = 0;
    Kept mine;
    uint32_t state = kAgain;
    float top = 0.0f, low = 0.0f;  // the interval of the collected, and what lies above it
    uint64_t above = 0u;
    for (int tries = 0; state == kAgain && tries < 4; ++tries) {
        uint64_t rough = 0u;
        if (team.rank == 0) {
            // A thread owns kPer neighbouring bins.
            constexpr int kPer = kBins / kThreads;
            uint64_t part[kPer], sum = 0u, all;
#pragma unroll
            for (int j = 0; j < kPer; ++j) part[j] = 0u;
#pragma unroll
            for (uint32_t c = 0; c < kMaxTeam; ++c) {
                if (c >= team.size) break;
                const uint4 *h = reinterpret_cast<const uint4 *>(team.peer(c)->hist) + threadIdx.x * (kPer / 4);
#pragma unroll
                for (int j = 0; j < kPer; j += 4) {
                    const uint4 v = h[j / 4];
                    part[j] += v.x, part[j + 1] += v.y, part[j + 2] += v.z, part[j + 3] += v.w;
                }
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                // in units of 2^-40 where that is the finer, and cut off there elsewhere
                const int up = 40 - bits - bin_power(threadIdx.x * kPer + j);
                if (MASS) part[j] = up >= 0 ? part[j] << up : part[j] >> -up;
                sum += part[j];
            }
            const uint64_t before = block_scan(sum, sm, all);
            const int64_t want = int64_t(target) - error;
            const uint64_t aim = want < 1 ? 1u : all < uint64_t(want) ? all : uint64_t(want);
            uint64_t at = before;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (at < aim && at + part[j] >= aim) sm.bin = threadIdx.x * kPer + j;
                at += part[j];
            }
            __syncthreads();
            const uint32_t lo = sm.bin > 0 ? sm.bin - 1 : 0;
            if (lo / kPer == threadIdx.x) {
                at = before;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (uint32_t(j) < lo % kPer) at += part[j];
                sm.above = at;
            }
            __syncthreads();
            rough = sm.above;
        }
        if (threadIdx.x == 0) {
            sm.count = 0u;
            sm.units = 0u;
        }
        team.sync();
        // Tokens of the cut's bin and its neighbours, as an interval of
        // values, to the list; those above it added up.
        const uint32_t bin = team.lead->bin, lo = bin > 0 ? bin - 1 : 0;
        const float unit = 1.0f / (kBinsPerPower * scale.power);
        top = bin > 1 ? scale.m - (float(lo) - 0.5f) * unit : 3.402823466e38f;
        low = fmaxf(scale.m - (float(bin) + 1.5f) * unit, -3.402823466e38f);
        mass = 0.0f;
        mine = Kept();
        row.each(sm, [&](const Piece<T, kVec> &x, const T *at, uint32_t i) {
            if (!__any_sync(kFull, piece_max(x) >= low)) return;
            float w[kVec];
            uint32_t list = 0u, sure = 0u;
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) {
                const float v = sample_value(row_to_float(x.v[e]));
                const bool in = v >= low && (!FLOOR || floor.keeps(v, i + e)), over = in && v > top;
                w[e] = scale.w(v);
                if (in && !over) list |= 1u << e;
                mass += over ? (MASS ? w[e] : 1.0f) : 0.0f;
                const bool keep = over && w[e] >= q;
                mine.sum += keep ? w[e] : 0.0f;
                if (keep) sure |= 1u << e;
            }
            team.append(list, at, i);
            if (kept && __any_sync(kFull, sure != 0u)) {
                float u[kVec];
                row.uniforms(i, u);
                // where one piece is kept the next is likely to be
                const uint32_t next = i + row.team * kVec;
                if (next < row.vocab) asm volatile("prefetch.global.L2 [%0];" ::"l"(row.u + next));
                mine.draw.offer(w, sure, u, row, scale, at, i);
            }
        });
        mass = team.sum(mass);  // past which every list is complete
        const uint32_t n = team.gather_lists();
        if (team.rank == 0) {
            // The cut is in the list if the tokens above it stay below the
            // target and the list reaches it.  A histogram leaves few to sort.
            above = MASS ? uint64_t(double(mass) * double(kFixed) + 0.5) : uint64_t(mass);
            error = int64_t(above) - int64_t(rough);
            auto amount = [&](uint64_t key) { return MASS ? scale.fixed(key_value(key)) : uint64_t(1); };
            auto keep = [&](uint64_t key) {  // its weight if it is kept
                const float w = scale.w(key_value(key));
                if (!kept || w < q) return 0.0f;
                if (w >= kLightest) mine.draw.take(w, row.u[key_index(key)], key_index(key));
                return w;
            };
            SubBin sub{0.0f, 0.0f, uint32_t(kSubBins), 0u};
            if (n <= kList && above < target) {
                const float first = fminf(top, scale.m);
                sub = sub_bin(sm, n, first, first - low, false, above, target, amount);
            }
            if (threadIdx.x == 0) sm.state = n <= kList ? kAgain : kMissed;
            if (sub.at < uint32_t(kSubBins)) {
                uint32_t few = pick_few(sm, n, [&](uint64_t key) { return sub.of(key) == sub.at; });
                const bool fits = few <= kFew;
                if (fits) {
                    // The list's order is not the same every time: added up in
                    // units, as the histogram has done if none is lighter than q.
                    const bool known = MASS && !(q > 0.0f);
                    uint64_t units = 0u;
                    for (uint32_t j = threadIdx.x; j < n; j += kThreads)
                        if (sub.of(sm.list[j]) < sub.at) {
                            const float w = keep(sm.list[j]);
                            if (!known) units += __float2ull_rn(w * kFixed);
                        }
                    if (!known) add_units(units, &sm.units);
                    else if (threadIdx.x == 0) sm.units = sub.before - above;
                }
                uint64_t *list = fits ? sm.few : sm.list;
                few = fits ? few : n;
                sort_list(list, few);
                const uint32_t per = (few + kThreads - 1) / kThreads;
                const uint32_t first = min(few, threadIdx.x * per), last = min(few, first + per);
                uint64_t sum = 0u, all;
                for (uint32_t j = first; j < last; ++j) sum += amount(list[j]);
                uint64_t before = (fits ? sub.before : above) + block_scan(sum, sm, all);
                for (uint32_t j = first; j < last && before < target; ++j) {
                    mine.sum += keep(list[j]);
                    before += amount(list[j]);
                    if (before >= target) {
                        sm.cut = list[j];
                        sm.state = kFound;
                    }
                }
            }
        }
        team.sync();
        state = team.lead->state;
        team.sync();  // everyone has read it, and the list may be filled anew
    }
    if (kept) {
        *kept = mine;
        if (team.rank == 0 && threadIdx.x == 0) kept->sum += from_fixed(sm.units);
    }
    if (state != kFound) {
        if (team.rank == 0) {
            // Among the interval's tokens where those were only too many (equal
            // values), else among all; and among all where the interval ends
            // before the cut, which the rounded amounts allow.
            const Row<T> whole(row.x, row.u, row.vocab, 0, 1);
            uint64_t cut = 0u;
            for (bool part = state == kMissed && above < target, on = true; on; part = false) {
                if (!part) {
                    top = 3.402823466e38f;
                    low = -top;
                    above = 0u;
                }
                cut = select_cut(target, above, sm, [&](auto add) {
                    whole.each(sm, [&](const Piece<T, kVec> &x, const T *, uint32_t i) {
                        if (!__any_sync(kFull, piece_max(x) >= low)) return;
#pragma unroll
                        for (uint32_t e = 0; e < kVec; ++e) {
                            const float v = sample_value(row_to_float(x.v[e]));
                            if (v >= low && v <= top && (!FLOOR || floor.keeps(v, i + e)))
                                add(order_key(v, i + e), MASS ? scale.fixed(v) : uint64_t(1));
                        }
                    });
                });
                on = cut == 0u && part;
            }
            __syncthreads();
            if (threadIdx.x == 0) sm.cut = cut;
        }
        team.sync();
    }
    cut_key = floor_key > team.lead->cut ? floor_key : team.lead->cut;
    team.sync();
    return state == kFound && kept != nullptr;
}

// The rest of a row whose n candidates, all tokens not below `threshold`, are
// in the leader's list, by the leader's CTA: top-k, top-p, min-p, draw.  A
// histogram of the list finds the first cut's bin, and few tokens are left to
// sort: with top-k those down to the bin, else the bin of the top-p cut alone,
// the tokens above it being kept as they are.  `total` is the sum of all
// tokens' weights where the list may not hold every one that has some; returns
// false, with nothing written, where the list then ends before the top-p cut.
__device__ __noinline__ bool finish_list(Smem &sm, uint32_t n, uint32_t k, float t, float p, float q, float threshold,
                                         float total, const float *__restrict__ u, int32_t *token, float *logprob)
{
    uint64_t *list = sm.list;
    Team alone(sm, 1);
    if (threadIdx.x == 0) sm.units = 0u;
    uint64_t most = 0u;
    for (uint32_t j = threadIdx.x; j < n; j += kThreads) most = list[j] > most ? list[j] : most;
    const Scale scale(key_value(alone.largest(most)), t);
    // Down to the threshold, or 32 t below the maximum, where no weight is left.
    const bool open = scale.m - 32.0f * t > threshold;
    const float span = scale.m - fmaxf(threshold, scale.m - 32.0f * t);
    Kept kept;
    float x = 0.0f;  // of the token that this thread would draw
    auto keep = [&](uint64_t key) {  // its weight if it is kept
        const uint32_t i = key_index(key);
        const float w = scale.w(key_value(key));
        if (w < q) return 0.0f;
        if (w < kLightest) return w;
        kept.draw.take(w, u[i], i);
        if (kept.draw.index == i) x = key_value(key);
        return w;
    };
    uint64_t before = 0u, target = ~uint64_t(0), sum = 0u, all;
    bool cut = false;  // top-p's target is known
    if (n > 64 && k < n) {
        const SubBin sub = sub_bin(sm, n, scale.m, span, open, 0u, k, [](uint64_t) { return uint64_t(1); });
        const uint32_t last = open ? min(sub.at, uint32_t(kSubBins - 2)) : sub.at;
        const uint32_t few = pick_few(sm, n, [&](uint64_t key) { return sub.of(key) <= last; });
        if (few <= kFew) {
            list = sm.few;
            n = few;
        }
    } else if (n > 64 && p < 1.0f) {
        for (uint32_t j = threadIdx.x; j < n; j += kThreads) sum += scale.fixed(key_value(list[j]));
        block_scan(sum, sm, all);
        const uint64_t aim = share_of(p, total > 0.0f ? double(total) * double(kFixed) : double(all));
        if (all < aim) return false;
        const SubBin sub = sub_bin(sm, n, scale.m, span, open, 0u, aim,
                                   [&](uint64_t key) { return scale.fixed(key_value(key)); });
        const uint32_t few = pick_few(sm, n, [&](uint64_t key) { return sub.of(key) == sub.at; });
        if (sub.at < uint32_t(kSubBins) && few <= kFew) {
            // added up in units, as in find_cut
            uint64_t units = 0u;
            for (uint32_t j = threadIdx.x; j < n; j += kThreads)
                if (sub.of(list[j]) < sub.at) {
                    const float w = keep(list[j]);
                    if (q > 0.0f) units += __float2ull_rn(w * kFixed);
                }
            if (q > 0.0f) add_units(units, &sm.units);
            else if (threadIdx.x == 0) sm.units = sub.before;
            list = sm.few;
            n = few;
            cut = true;
            target = aim;
            before = sub.before;
        }
    }
    for (uint32_t j = threadIdx.x; j < n; j += kThreads)  // on their way while the list is sorted
        asm volatile("prefetch.global.L2 [%0];" ::"l"(u + key_index(list[j])));
    sort_list(list, n);
    n = min(k, n);
    const uint32_t per = (n + kThreads - 1) / kThreads;
    const uint32_t first = min(n, threadIdx.x * per), last = min(n, first + per);
    if (p < 1.0f) {
        sum = 0u;
        for (uint32_t j = first; j < last; ++j) sum += scale.fixed(key_value(list[j]));
        before += block_scan(sum, sm, all);
        if (!cut) target = share_of(p, total > 0.0f ? double(total) * double(kFixed) : double(all));
        if (!cut && all < target) return false;
    }
    for (uint32_t j = first; j < last && before < target; ++j) {
        kept.sum += keep(list[j]);
        if (p < 1.0f) before += scale.fixed(key_value(list[j]));
    }
    if (threadIdx.x == 0) kept.sum += from_fixed(sm.units);  // past sort_list's barriers
    const KeySum end = alone.reduce(KeySum{kept.draw.key(), kept.sum});
    if (kept.draw.key() == end.key) {
        *token = int32_t(key_index(end.key));
        if (logprob) *logprob = scale.z(x) - logf(end.sum);
    }
    return true;
}

// A value that about k in kBatch of the row's tokens are not below: the k-th
// largest of the threads' maxima over the CTA's first kBatch tokens, rounded
// down to 16 bits.
template <class T>
__device__ __forceinline__ float sample_bound(const Row<T> &row, uint32_t k)
{
    constexpr uint32_t kVec = Row<T>::kVec;
    float best = -INFINITY;
#pragma unroll
    for (int b = 0; b < kSample; b += kSample / 2) {
        Piece<T, kVec> pc[kSample / 2];
#pragma unroll
        for (int j = 0; j < kSample / 2; ++j) row.load((b + j) * row.team + row.me, pc[j]);
#pragma unroll
        for (int j = 0; j < kSample / 2; ++j) best = fmaxf(best, piece_max(pc[j]));
    }
    const uint32_t least = kth_largest(best > -INFINITY ? order_bits(sample_value(best)) : 0u, k);
    return least ? order_value(least) : -INFINITY;
}

// The tokens from the cut on that weigh at least q: the sum of their weights
// and the draw, this thread's share.
template <class T>
__device__ __noinline__ Kept draw_row(const Team &team, const Row<T> &row, const Scale &row_scale, uint64_t cut_key,
                                      float q)
{
    constexpr uint32_t kVec = Row<T>::kVec;
    Kept kept;
    const Scale scale = row_scale;
    const Cut cut(cut_key);
    row.each(team.sm, [&](const Piece<T, kVec> &x, const T *at, uint32_t i) {
        float w[kVec], u[kVec];
        uint32_t in = 0u;
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) {
            const float v = sample_value(row_to_float(x.v[e]));
            w[e] = scale.w(v);
            if (w[e] >= q && w[e] > 0.0f && cut.keeps(v, i + e)) in |= 1u << e;
        }
        if (!__any_sync(kFull, in != 0u)) return;
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) kept.sum += (in >> e) & 1u ? w[e] : 0.0f;
        row.uniforms(i, u);
        kept.draw.offer(w, in, u, row, scale, at, i);
    });
    return kept;
}

// The same of all tokens, whose u are all needed and come with the logits.
template <class T>
__device__ __noinline__ Kept draw_all(const Team &team, const Row<T> &row, const Scale &row_scale)
{
    constexpr uint32_t kVec = Row<T>::kVec;
    Kept kept;
    const Scale scale = row_scale;
    row.template each<true>(team.sm, [&](const Piece<T, kVec> &x, const T *at, uint32_t i, const float4 *us) {
        float w[kVec], u[kVec];
        uint32_t in = 0u;
#pragma unroll
        for (uint32_t e = 0; e < kVec; e += 4) {
            const float4 r = us[e / 4 * kThreads];
            u[e] = r.x, u[e + 1] = r.y, u[e + 2] = r.z, u[e + 3] = r.w;
        }
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) {
            w[e] = scale.w(sample_value(row_to_float(x.v[e])));
            kept.sum += w[e];
            if (w[e] > 0.0f) in |= 1u << e;
        }
        kept.draw.offer(w, in, u, row, scale, at, i);
    });
    return kept;
}

template <class T>
__global__ void __launch_bounds__(kThreads, kResident)
sample_kernel(const T *__restrict__ logits, size_t logits_stride, uint32_t vocab,
              const float *__restrict__ uniform, size_t uniform_stride, const float *__restrict__ temperature,
              const int32_t *__restrict__ top_k, const float *__restrict__ top_p, const float *__restrict__ min_p,
              int32_t *__restrict__ tokens, float *__restrict__ logprobs)
{
    extern __shared__ __align__(16) uint8_t sample_smem[];
    Smem &sm = *reinterpret_cast<Smem *>(sample_smem);
    constexpr uint32_t kVec = Row<T>::kVec;
    Team team(sm, cg::this_cluster().num_blocks());
    if (threadIdx.x == 0) sm.count = 0u;
    team.started();
    const uint32_t r = blockIdx.x / team.size;
    const Row<T> row(logits + size_t(r) * logits_stride, uniform + size_t(r) * uniform_stride, vocab, team.rank,
                     team.size);
    const float t = temperature ? temperature[r] : 1.0f;
    const float p = top_p ? top_p[r] : 1.0f;
    const float q0 = min_p ? min_p[r] : 0.0f, q = q0 > 0.0f ? fminf(q0, 1.0f) : 0.0f;
    const bool greedy = uniform == nullptr || !(t > 0.0f);
    const uint32_t k = top_k && top_k[r] > 0 ? min(uint32_t(top_k[r]), vocab) : vocab;
    int32_t *token = tokens + r;
    float *logprob = logprobs ? logprobs + r : nullptr;
    team.all_started();

    // By one pass that collects candidates: all tokens of a short row (one of
    // 4000 with top-p 0.9: 18 us); with a small top-k those not below a bound,
    // the k-th largest of the threads' maxima over each CTA's first kBatch
    // tokens, rounded down to 16 bits (7 us; 12 where all are listed). About k in
    // kBatch tokens get in; at k = kThreads / 2, -512 ln(1 - 1/2) = 355 a batch,
    // which a list has room for.
    constexpr uint32_t kBatch = kSample * kThreads * kVec;
    const bool brief = vocab <= kList && (k == vocab || k <= kFew / 2);
    if (!greedy && (k < vocab || p < 1.0f) &&
        (brief || (k <= uint32_t(kThreads / 2) && uint64_t(k) * vocab <= uint64_t(kBatch) * (kList / 2)))) {
        float threshold = -INFINITY;
        if (!brief || (k <= uint32_t(kThreads / 2) && vocab > uint32_t(kFew))) threshold = sample_bound(row, k);
        threshold = fmaxf(threshold, -3.402823466e38f);  // -inf is no candidate
        row.each(sm, [&](const Piece<T, kVec> &x, const T *at, uint32_t i) {
            if (!__any_sync(kFull, piece_max(x) >= threshold)) return;
            uint32_t which = 0u;
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e)
                if (row_to_float(x.v[e]) >= threshold) which |= 1u << e;
            team.append(which, at, i);
        });
        team.sync();
        const uint32_t n = team.gather_lists();
        team.sync();  // the leader has read every list, and counts anew
        if (n <= kList) {
            if (team.rank == 0) {
                if (n > 0) {
                    finish_list(sm, n, k, t, p, q, threshold, 0.0f, row.u, token, logprob);
                } else if (threadIdx.x == 0) {
                    *token = -1;
                    if (logprob) *logprob = -INFINITY;
                }
            }
            return;  // nobody reads another CTA's shared memory any more
        }
    }

    // Without a filter nothing needs the maximum: any token near it serves as
    // the weights' unit, and one pass is enough unless they come out too large.
    if (!greedy && k == vocab && p >= 1.0f && q == 0.0f) {
        Piece<T, kVec> pc;
        row.load(row.me, pc);
        const float near = sample_value(piece_max(pc));
        const uint64_t unit = team.largest(near > -INFINITY ? order_key(near, 0u) : 0u);
        if (unit != 0u) {
            const Scale scale(key_value(unit), t);
            const Kept kept = draw_all(team, row, scale);
            const KeySum end = team.reduce(KeySum{kept.draw.key(), kept.sum});
            if (end.sum < 1e30f) {
                if (team.rank == 0 && threadIdx.x == 0) {
                    const uint32_t i = key_index(end.key);
                    *token = int32_t(i);
                    // z and log(sum) are far from 0 where the unit is far from the
                    // maximum; the quotient does not lose what they share
                    if (logprob) *logprob = fminf(logf(scale.w(row.value(i)) / end.sum), 0.0f);
                }
                team.sync();  // no CTA leaves while another may write to its slots
                return;
            }
        }
    }

    // The first of the order.  Where top-p stands alone and a CTA has a row, the
    // same pass lists the largest tokens and adds up all weights, in units of the
    // thread's maximum so far: the cut of a row with a few likely tokens is in
    // the list, and the row is done.  512 x 128000 float32, normal logits with 40
    // raised by up to 12, against the passes below alone: T = 0.5, p = 0.95 143 us
    // for 266; T = 0.7, p = 0.9 244 for 295; where no list holds the cut, T = 1,
    // p = 0.95 444 for 385 and T = 1.2 453 for 391 (304 x 128000 bf16: 68 for 129,
    // 147 for 154, 203 for 174 and 203 for 172).  Which it will be shows in the row
    // alone.  Not for rows of a few samples (200 x 20000: 33 us for 49, but 70 for
    // 55), nor for few rows, whose time is that of the barriers.
    const uint32_t wish = min(uint32_t(kThreads / 2), uint32_t(uint64_t(kBatch) * (kList / 2) / vocab));
    const bool likely =
        !greedy && k == vocab && p < 1.0f && team.size == 1 && vocab >= 3u * kBatch && wish >= 32u;
    float threshold = INFINITY, unit = -3.402823466e38f, total = 0.0f;
    const float power = Scale(0.0f, t).power;
    if (likely) {
        if (threadIdx.x == 0) sm.count = 0u;
        threshold = fmaxf(sample_bound(row, wish), -3.402823466e38f);
        __syncthreads();
    }
    float best = -INFINITY;
    uint32_t at = ~0u;
    row.each(sm, [&](const Piece<T, kVec> &x, const T *p, uint32_t i) {
        const float top = sample_value(piece_max(x));
        if (likely) {
            if (top > unit) {
                total *= exp2f((unit - top) * power);
                unit = top;
            }
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) total += exp2f((sample_value(row_to_float(x.v[e])) - unit) * power);
            if (__any_sync(kFull, top >= threshold)) {
                uint32_t which = 0u;
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e)
                    if (row_to_float(x.v[e]) >= threshold) which |= 1u << e;
                team.append(which, p, i);
            }
        }
        if (top > best || (top == best && i < at)) {
            best = top;
            for (int e = int(kVec) - 1; e >= 0; --e)
                if (sample_value(row_to_float(p[e])) == top) at = i + e;
        }
    });
    const uint64_t first = team.largest(best > -INFINITY ? order_key(best, at) : 0u);
    if (first == 0u || greedy) {
        if (team.rank == 0 && threadIdx.x == 0) {
            *token = first == 0u ? -1 : int32_t(key_index(first));
            if (logprob) *logprob = first == 0u ? -INFINITY : 0.0f;
        }
        team.sync();  // no CTA leaves while another may write to its slots
        return;
    }
    const Scale scale(key_value(first), t);
    if (likely) {
        total = team.sum(total * scale.w(unit));
        const uint32_t n = sm.count;
        __syncthreads();
        if (n <= kList && finish_list(sm, n, k, t, p, q, threshold, total, row.u, token, logprob)) return;
        __syncthreads();
    }
    Kept kept;
    uint64_t cut_key = 0u;
    bool done = false;
    if (k < vocab) done = find_cut<false, false>(team, row, scale, 0u, k, 1.0f, q, p < 1.0f ? nullptr : &kept, cut_key);
    if (p < 1.0f)
        done = cut_key ? find_cut<true, true>(team, row, scale, cut_key, 0u, p, q, &kept, cut_key)
                       : find_cut<true, false>(team, row, scale, 0u, 0u, p, q, &kept, cut_key);
    if (!done) kept = draw_row(team, row, scale, cut_key, q);
    const KeySum end = team.reduce(KeySum{kept.draw.key(), kept.sum});
    if (team.rank == 0 && threadIdx.x == 0) {
        const uint32_t i = key_index(end.key);
        *token = int32_t(i);
        if (logprob) *logprob = scale.z(row.value(i)) - logf(end.sum);
    }
    team.sync();  // no CTA leaves while another may write to its slots
}

template <class T, class... A>
cudaError_t run_sample(const void *logits, uint32_t rows, uint32_t vocab, cudaStream_t s, size_t stride, A... args)
{
    // Few rows are spread over more CTAs, down to two pieces per thread: one row
    // of 128000 bf16 with top-p 0.95 takes 53 us by eight CTAs, 67 by four.
    // With more rows than that one CTA each is best (above).
    const uint64_t slots = uint64_t(kResident) * uint64_t(gch::sm_count());
    uint32_t team = 1;
    while (team < kMaxTeam && uint64_t(rows) * (2 * team) <= slots &&
           vocab >= 2 * team * (kThreads * 2 * uint32_t(16 / sizeof(T))))
        team *= 2;
    // Raises the kernel's shared-memory limit, once per device.
    auto kernel = sample_kernel<T>;
    if (gch::persistent_grid(reinterpret_cast<const void *>(kernel), kThreads, sizeof(Smem), 1) <= 0)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rows * team);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = team;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(logits), stride, vocab, args...);
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
