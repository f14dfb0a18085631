// verify.cu -- drafted tokens accepted or replaced against the target's
// probabilities, from given uniform random numbers (gc_sample_verify).
//
// Per sequence, with p the softmax of the target's row of a position at the
// sequence's temperature, q the draft's, d the drafted token and u its random
// number: positions are accepted while u q(d) < p(d).  At the first that is not
// the token is drawn from max(p - q, 0), past the last draft from p: the
// largest r / -log v over the tokens, v their random numbers, which is a draw
// with probability r / sum r.
//
// Two launches.  The first takes every row in chunks, one CTA each, and leaves
// each chunk's maximum m and sum of exp((x - m) / T) (greedy sequences: the
// first of the largest values).  The second reads one row of each sequence
// again, the one at which it stops, and draws.  Chunks go by position first,
// then by sequence: where there are many more than the GPU holds at a time, the
// last chunk of a position decides it, and chunks of later positions of a
// sequence that has stopped are not read.
//
// exp((x - m) / T) is 2^(x f - c) with f = log2(e) / T and c = m f rounded: one
// multiply-add, whose only rounding is that of the exponent, since every weight
// of a row carries the same 2^(m f - c) and p is a quotient of them.
//
// Measured, kernels alone: 192 sequences of 5 drafts by a model, 128000 bf16, four
// in five positions accepted: 119 us.  The rows take 72 of it, 356 MB at 5.1 TB/s,
// where 316 MB would do (the rest was under way when its sequence stopped), bound
// by instructions: 11 a logit, 79 to 87% of the issue slots (of 48 and 96
// sequences), 35% of the pipe of exponentials.  The draw takes 46: 98 MB of
// random numbers and two rows of each sequence once more.  Where filters have
// left 50 tokens of each row, 146 us, 15 instructions a logit (rare_piece), against
// 123 of the same rows whole; greedy sequences 62.  One sequence of 4 drafts, 32768
// float32: 12 us, two launches' chains of dependent reads.
#include <atomic>

#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRing = 6;              // pieces of 16 bytes that a thread has under way
constexpr int kAtOnce = 2;            // of them waited for and loaded again together
constexpr int kDrawRing = 3;          // pieces of each of three rows in the draw
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLargest = 3.402823466e38f;
constexpr float kUniformLo = 0x1p-25f, kUniformHi = 1.0f - 0x1p-24f;

// Chunks: 16 pieces per thread, 64 KB (8 a thread take 131 us at the size above,
// for what every CTA does once; 32 take 118, with 50 MB more under way), where that makes more CTAs than the
// GPU holds, else fewer.
constexpr uint32_t kDrawWave = 4;  // CTAs per SM of the draw
constexpr uint32_t kSteps = 16, kWave = 6;  // kWave: CTAs per SM of the rows
// Positions are decided on the way where chunks are more than this many times
// what the GPU holds at a time.  Of 5 drafts of 128000 bf16, 32 sequences take 43 us
// so and 38 without, 96 take 76 and 76, 128 take 89 and 96, 192 take 120 and 136.
constexpr size_t kSkipWaves = 5;

// z = (x - m) / t as a power of two's exponent.
__device__ __forceinline__ float power_of(float t)
{
    return fminf(fmaxf(1.0f / t, 1.17549435e-38f) * 1.44269504f, kLargest);
}

__device__ __forceinline__ uint64_t first_key(float x, uint32_t i)
{
    return (uint64_t(order_bits(x)) << 32) | uint32_t(~i);
}

// A chunk's or a row's maximum and sum; of greedy sequences the key of the
// first of the largest values.
union Part {
    struct {
        float m, sum;
    };
    uint64_t key;
};
static_assert(sizeof(Part) == 8, "Part");

struct Verify {
    uint32_t sequences, drafts, vocab;
    size_t x_stride, d_stride, u_stride;
    const void *x, *d;          // target and draft logits; d may be NULL
    const int32_t *ids;         // drafted tokens
    const float *accept, *uniform, *temperature;
    int32_t *tokens, *accepted;
    float *logprobs;
    // workspace
    uint32_t chunk, chunks;     // pieces in a chunk, chunks of a row
    Part *x_part, *d_part;      // [row][chunk]
    unsigned long long *best;   // per sequence: the draw so far
    uint32_t *drawn;            // per sequence: chunks that have drawn
    uint32_t *left, *arrived;   // per sequence: drafts from the first rejected one on; per position: chunks done; NULL: not kept
    uint32_t draw, draws;       // pieces in a chunk of the draw, chunks

    // without random numbers every sequence is greedy
    __device__ __forceinline__ float t(uint32_t b) const
    {
        return uniform == nullptr ? 0.0f : temperature ? temperature[b] : 1.0f;
    }
    __device__ __forceinline__ bool real(uint32_t id) const { return id < vocab; }
};

// A row's pieces of 16 bytes from the first aligned element on; the elements
// before and after them are single.
template <class T>
struct Pieces {
    static constexpr uint32_t kVec = 16 / sizeof(T);
    const T *x;
    uint32_t head, count, vocab;
    __device__ __forceinline__ Pieces(const T *x_, uint32_t vocab_) : x(x_), vocab(vocab_)
    {
        const uint32_t lead = uint32_t((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / uint32_t(sizeof(T));
        head = min(lead, vocab);
        count = (vocab - head) / kVec;
    }
    // Thread i's single element, or vocab.
    __device__ __forceinline__ uint32_t single(uint32_t i) const
    {
        const uint32_t tail = head + count * kVec;
        if (i < head) return i;
        return i - head < vocab - tail ? tail + (i - head) : vocab;
    }
};

// Whether c = m * power can be taken off by a multiply-add: every weight then
// carries 2^(m * power - c), which has to stay near 1.
__device__ __forceinline__ bool plain(float c) { return fabsf(c) < 0x1p24f; }

// The weight of a logit by a maximum, of any values.
__device__ __forceinline__ float weight(float x, float m, float power)
{
    x = sample_value(x);
    const float c = m * power;
    return pow2(plain(c) ? fmaf(x, power, -c) : (x - m) * power);
}

// m and sum joined with another maximum and sum.  Each sum's weights are by its
// own m: less c where that is plain, less the exact product where not.
__device__ __forceinline__ void join(float &m, float &sum, float m2, float sum2, float power)
{
    const float top = fmaxf(m, m2);
    if (!(top > -INFINITY)) return;
    auto scale = [&](float from) {
        const float c = from * power, d = top * power;
        if (plain(c)) return pow2(plain(d) ? c - d : fmaf(-top, power, c));
        return pow2(plain(d) ? fmaf(from, power, -d) : (from - top) * power);
    };
    sum = (m == top ? sum : sum * scale(m)) + (m2 == top ? sum2 : sum2 * scale(m2));
    m = top;
}

// m and sum of all lanes, to all of them.
__device__ __forceinline__ void join_lanes(float &m, float &sum, float power)
{
    const uint32_t bits = __reduce_max_sync(kFull, order_bits(m));
    float top = order_value(bits), s = 0.0f;
    if (top > -INFINITY) {
        join(top, s, m, sum, power);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    }
    m = top, sum = s;
}

__device__ __forceinline__ void copy_piece(void *to, const void *from, bool there)
{
    if (there)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from)
                     : "memory");
}

__device__ __forceinline__ void copy_float(void *to, const float *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
}

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A chunk's pieces to f, one after another, through a ring of asynchronous
// copies, each thread its own: kRing of them are under way at any time.  A round
// of the ring is unrolled, so that its places and the copies' addresses are
// constants.
template <class T, class F>
__device__ __forceinline__ void each_piece(const Pieces<T> &row, uint32_t first, uint32_t end, uint4 *ring, const F &f)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    const uint32_t j = first + threadIdx.x;
    const int left = j < end ? int((end - j + kThreads - 1) / kThreads) : 0;  // of this thread
    const T *from = row.x + row.head + size_t(j) * kVec;
    uint32_t at = row.head + j * kVec;
    uint4 *mine = ring + threadIdx.x;
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
        copy_piece(mine + q * kThreads, from + q * kThreads * kVec, q < left);
        if (q % kAtOnce == kAtOnce - 1) commit_copies();
    }
    for (int i = 0; i < left; i += kRing) {
        from += kRing * kThreads * kVec;
#pragma unroll
        for (int q = 0; q < kRing; ++q) {
            if (q % kAtOnce == 0) wait_copies<kRing / kAtOnce - 1>();
            if (i + q < left) f(mine + q * kThreads, at + q * kThreads * kVec);
            copy_piece(mine + q * kThreads, from + q * kThreads * kVec, i + q + kRing < left);
            if (q % kAtOnce == kAtOnce - 1) commit_copies();
        }
        at += kRing * kThreads * kVec;
    }
    wait_copies<0>();
}

// A piece that holds a thread's first open logits (or, before them, none), a NaN,
// an infinity or a logit far above m: the new (m, sum).  Out of line, with the
// piece still in shared memory.
template <class T>
__device__ __noinline__ float2 rare_piece(const uint4 *at, float m, float sum, float power)
{
    constexpr int kVec = 16 / sizeof(T);
    float x[kVec];
    piece_values(load_piece<T, kVec>(reinterpret_cast<const T *>(at)), x);
    float top = m;
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = fmaxf(top, x[e]);
    top = fminf(top, kLargest);
    if (top > -INFINITY) {
        join(m, sum, top, 0.0f, power);
#pragma unroll 1
        for (int e = 0; e < kVec; ++e) sum += weight(row_to_float(reinterpret_cast<const T *>(at)[e]), m, power);
    }
    return make_float2(m, sum);
}

// A chunk's sum by a maximum, to lane 0 of warp 0.  The maximum is one of the
// chunk's first logits: later ones may weigh up to 2^60, which spares looking
// for the largest.
template <class T>
__device__ __forceinline__ Part chunk_sum(const Pieces<T> &row, uint32_t first, uint32_t end, bool singles, float power,
                                          uint4 *ring, Part *s_part)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    float m = -INFINITY, sum = 0.0f, c = INFINITY;  // no reference yet: the first piece is rare
    each_piece(row, first, end, ring, [&](const uint4 *at, uint32_t) {
        float x[kVec], more = 0.0f;
        piece_values(load_piece<T, kVec>(reinterpret_cast<const T *>(at)), x);
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) more += pow2(fmaf(x[e], power, -c));
        if (more <= 0x1p60f && c < INFINITY) {
            sum += more;
        } else {
            const float2 r = rare_piece<T>(at, m, sum, power);
            m = r.x, sum = r.y;
            c = m > -INFINITY && plain(m * power) ? m * power : INFINITY;
        }
    });
    if (singles) {
        const uint32_t i = row.single(threadIdx.x);
        if (i < row.vocab) {
            // by itself, with the rounding that its own product with `power` leaves in every weight by it
            const float x = sample_value(row_to_float(row.x[i]));
            if (x > -INFINITY) join(m, sum, x, weight(x, x, power), power);
        }
    }
    join_lanes(m, sum, power);
    Part p;
    p.m = m, p.sum = sum;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = p;
    __syncthreads();
    if (threadIdx.x < 32) {
        const bool has = threadIdx.x < kWarps;
        m = has ? s_part[threadIdx.x].m : -INFINITY, sum = has ? s_part[threadIdx.x].sum : 0.0f;
        join_lanes(m, sum, power);
        p.m = m, p.sum = sum;
    }
    return p;
}

// The key of the first of a chunk's largest values, to lane 0 of warp 0.
template <class T>
__device__ __forceinline__ Part chunk_first(const Pieces<T> &row, uint32_t first, uint32_t end, bool singles,
                                            uint4 *ring, Part *s_part)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    uint64_t key = first_key(-INFINITY, ~0u);
    float top = -INFINITY;
    each_piece(row, first, end, ring, [&](const uint4 *at, uint32_t i) {
        const Piece<T, kVec> v = load_piece<T, kVec>(reinterpret_cast<const T *>(at));
        if (!(piece_max(v) > top)) return;  // a thread's pieces come in order: equal values later count for nothing
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) {
            const float x = sample_value(row_to_float(v.v[e]));
            if (x > top) {
                top = x;
                key = first_key(x, i + e);
            }
        }
    });
    if (singles) {
        const uint32_t i = row.single(threadIdx.x);
        if (i < row.vocab) {
            const uint64_t k = first_key(sample_value(row_to_float(row.x[i])), i);
            key = k > key ? k : key;
        }
    }
    auto reduce = [&](uint32_t mask, int o) {
        for (; o > 0; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(mask, key, o);
            key = k > key ? k : key;
        }
    };
    reduce(kFull, 16);
    Part p;
    p.key = key;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = p;
    __syncthreads();
    if (threadIdx.x < kWarps) {
        key = s_part[threadIdx.x].key;
        reduce(0xffu, kWarps / 2);
        p.key = key;
    }
    return p;
}

// A row's parts joined by one warp; all lanes have the result.
__device__ __forceinline__ Part row_part(const Part *parts, uint32_t chunks, bool greedy, float power)
{
    const uint32_t lane = threadIdx.x & 31;
    Part r;
    if (greedy) {
        uint64_t key = 0;
        for (uint32_t c = lane; c < chunks; c += 32) {
            const uint64_t k = __ldcg(reinterpret_cast<const unsigned long long *>(parts + c));
            key = k > key ? k : key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(kFull, key, o);
            key = k > key ? k : key;
        }
        r.key = key;
        return r;
    }
    float m = -INFINITY, sum = 0.0f;
    for (uint32_t c = lane; c < chunks; c += 32) {
        Part p;
        p.key = __ldcg(reinterpret_cast<const unsigned long long *>(parts + c));
        join(m, sum, p.m, p.sum, power);
    }
    join_lanes(m, sum, power);
    r.m = m, r.sum = sum;
    return r;
}

// Whether position j < drafts of sequence b is accepted, by one warp; the rows'
// joined parts come along.
template <class T>
__device__ __forceinline__ bool decide(const Verify &a, uint32_t b, uint32_t j, Part &target, Part &draft)
{
    const float t = a.t(b), power = power_of(t);
    const bool greedy = !(t > 0.0f);
    const size_t row = size_t(b) * (a.drafts + 1) + j, at = size_t(b) * a.drafts + j;
    target = row_part(a.x_part + row * a.chunks, a.chunks, greedy, power);
    draft.m = 0.0f, draft.sum = 1.0f;
    if (j >= a.drafts) return false;
    const uint32_t id = uint32_t(a.ids[at]);
    if (!a.real(id)) return false;
    if (greedy) return uint32_t(target.key >> 32) > order_bits(-INFINITY) && uint32_t(~target.key) == id;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    // u q < p, with p = w / sum: in 64 bits, where the products are exact enough
    const double wp = weight(row_to_float(x[id]), target.m, power);
    double wq = 1.0;
    if (a.d) {
        draft = row_part(a.d_part + at * a.chunks, a.chunks, false, power);
        const T *d = static_cast<const T *>(a.d) + at * a.d_stride;
        wq = draft.sum > 0.0f ? weight(row_to_float(d[id]), draft.m, power) : 0.0f;
    }
    const double u = fminf(fmaxf(a.accept[at], kUniformLo), kUniformHi);
    return target.sum > 0.0f && u * wq * double(target.sum) < wp * (draft.sum > 0.0f ? double(draft.sum) : 1.0);
}

// One chunk of one row.
template <class T>
__global__ void __launch_bounds__(kThreads, kWave)
verify_rows_kernel(Verify a)
{
    __shared__ Part s_part[kWarps];
    __shared__ uint4 s_ring[kRing * kThreads];
    chain_start();
    // positions first, then chunks, sequences, target or draft
    const uint32_t j = blockIdx.z, c = blockIdx.y, kinds = a.d ? 2 : 1;
    const uint32_t kind = a.d ? blockIdx.x & 1u : 0u, b = a.d ? blockIdx.x >> 1 : blockIdx.x;
    if (kind == 1 && j == a.drafts) return;
    const int32_t *ids = a.ids + size_t(b) * a.drafts;
    if (a.left == nullptr) {
        if (j == 0 && kind == 0 && c == 0 && threadIdx.x == 0) {
            a.best[b] = 0;
            a.drawn[b] = 0;
        }
    } else if (__syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile uint32_t *>(a.left + b) > a.drafts - j)) {
        return;  // read once: the word may change between two threads' reads
    }
    const float t = a.t(b), power = power_of(t);
    const bool greedy = !(t > 0.0f);
    if (kind == 1 && greedy) return;
    // a position past the first drafted token that is none is not reached
    bool none = false;
    for (uint32_t i = threadIdx.x & 31; i < j + kind; i += 32) none |= !a.real(uint32_t(ids[i]));
    if (__any_sync(kFull, none)) return;

    const T *x = kind == 0 ? static_cast<const T *>(a.x) + (size_t(b) * (a.drafts + 1) + j) * a.x_stride
                           : static_cast<const T *>(a.d) + (size_t(b) * a.drafts + j) * a.d_stride;
    const Pieces<T> row(x, a.vocab);
    const uint32_t first = min(c * a.chunk, row.count), end = min(first + a.chunk, row.count);
    const Part p = greedy ? chunk_first(row, first, end, c == 0, s_ring, s_part)
                          : chunk_sum(row, first, end, c == 0, power, s_ring, s_part);
    Part *to = kind == 0 ? a.x_part + (size_t(b) * (a.drafts + 1) + j) * a.chunks + c
                         : a.d_part + (size_t(b) * a.drafts + j) * a.chunks + c;
    if (threadIdx.x == 0) to->key = p.key;
    if (a.left == nullptr || j == a.drafts || threadIdx.x >= 32) return;
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        before = atomicAdd(a.arrived + size_t(b) * a.drafts + j, 1u);
        __threadfence();
    }
    before = __shfl_sync(kFull, before, 0);
    __syncwarp();  // a shuffle orders nothing: the other lanes read the parts behind lane 0's fence
    none = !a.real(uint32_t(ids[j]));  // then the draft's row is not read
    if (before + 1 != a.chunks * (greedy || none ? 1 : kinds)) return;
    Part target, draft;
    if (!decide<T>(a, b, j, target, draft) && threadIdx.x == 0) atomicMax(a.left + b, a.drafts - j);
}

// Of the tokens offered, the largest r / -log v; equal ones, the lowest index.
// A token can only be it if -log v < r / bound for any ratio `bound` already
// seen, so v > 1 - r / bound: one multiply-add spares most tokens the logarithm.
// v is one that counts: numbers below 2^-25 and NaN are 2^-25.
struct Best {
    float ratio = 0.0f;
    uint32_t index = ~0u;
    float bound = 0.0f, slope = -kLargest;  // bound: the warp's; slope: -1 / bound and a little more
    __device__ __forceinline__ bool open(float r, float v) const { return !(v < fmaf(r, slope, 0.9999995f)); }
    __device__ __forceinline__ void take(float r, float v, uint32_t i)
    {
        if (!(r > 0.0f)) return;
        const float q = r / -logf(fminf(fmaxf(v, kUniformLo), kUniformHi));
        if (q > ratio || (q == ratio && i < index)) {
            ratio = q;
            index = i;
        }
    }
    // All lanes together: the bound of the warp.  Ratios are not negative, so
    // their bits are in order.
    __device__ __forceinline__ void share()
    {
        const float b = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(ratio)));
        if (b > bound) {
            bound = b;
            slope = -1.000001f / b;
        }
    }
    __device__ __forceinline__ uint64_t key() const
    {
        return ratio > 0.0f ? (uint64_t(__float_as_uint(ratio)) << 32) | uint32_t(~index) : 0;
    }
};

// The row at which a sequence stops, as its draw sees it.
template <class T>
struct Stop {
    const T *x, *d;     // d: NULL where nothing is taken off
    const float *u;
    float m, inverse, dm, dinverse, power, c, dc;
    uint32_t without;   // a token that cannot be drawn
    bool usual;         // multiply-adds do: no infinities

    // p - q.  A NaN of the draft weighs nothing; one of the target makes a NaN,
    // which is never taken.
    __device__ __forceinline__ float usual_r(float v, float w) const
    {
        const float p = pow2(__fmaf_rn(v, power, -c)), q = pow2(__fmaf_rn(w, power, -dc));
        return __fmaf_rn(fmaxf(q, 0.0f), -dinverse, __fmul_rn(p, inverse));
    }
    __device__ __forceinline__ float r(float v, float w) const
    {
        if (usual) return usual_r(v, w);
        return __fmaf_rn(weight(w, dm, power), -dinverse, __fmul_rn(weight(v, m, power), inverse));
    }
    __device__ __forceinline__ float r(uint32_t i) const
    {
        return r(row_to_float(x[i]), d ? row_to_float(d[i]) : -INFINITY);
    }
};

// The rings of the draw, in shared memory.
template <class T>
struct DrawRing {
    static constexpr int kWords = 4 / sizeof(T);  // of 16 bytes of random numbers per piece
    uint4 x[kDrawRing][kThreads], d[kDrawRing][kThreads];
    float4 u[kDrawRing][kWords][kThreads];
};

// Every thread of the CTA takes part.  Tokens that can win are few, and are
// read once more, so that their code is there once.
template <class T>
__device__ __forceinline__ Best chunk_draw(const Stop<T> &s, const Pieces<T> &row, uint32_t first, uint32_t end,
                                           bool singles, DrawRing<T> &ring)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    Best best;
    const bool d_whole = s.d && ((reinterpret_cast<uintptr_t>(s.d + row.head)) & 15u) == 0;
    const bool u_whole = ((reinterpret_cast<uintptr_t>(s.u + row.head)) & 15u) == 0;
    uint32_t lone = singles ? row.single(threadIdx.x) : row.vocab;
    auto copy = [&](uint32_t j, int slot) {
        if (j < end) {
            const uint32_t i = row.head + j * kVec;
            copy_piece(&ring.x[slot][threadIdx.x], s.x + i, true);
            copy_piece(&ring.d[slot][threadIdx.x], s.d + i, d_whole);
#pragma unroll
            for (int q = 0; q < DrawRing<T>::kWords; ++q) {
                float4 *to = &ring.u[slot][q][threadIdx.x];
                if (u_whole) {
                    copy_piece(to, s.u + i + 4 * q, true);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) copy_float(reinterpret_cast<float *>(to) + e, s.u + i + 4 * q + e);
                }
            }
        }
        commit_copies();
    };
#pragma unroll
    for (int q = 0; q < kDrawRing; ++q) copy(first + threadIdx.x + q * kThreads, q);
    int slot = 0;
    for (uint32_t base = first;; base += kThreads) {
        const uint32_t j = base + threadIdx.x, i = row.head + j * kVec;
        float r[kVec], u[kVec];
        uint32_t which = 0;
        wait_copies<kDrawRing - 1>();
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) r[e] = u[e] = 0.0f;
        if (j < end) {
            const Piece<T, kVec> v = load_piece<T, kVec>(reinterpret_cast<const T *>(&ring.x[slot][threadIdx.x]));
            Piece<T, kVec> w;
            if (d_whole) {
                w = load_piece<T, kVec>(reinterpret_cast<const T *>(&ring.d[slot][threadIdx.x]));
            } else {
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) w.v[e] = s.d ? s.d[i + e] : row_from_float<T>(-INFINITY);
            }
#pragma unroll
            for (uint32_t e = 0; e < kVec; e += 4) {
                const float4 f = ring.u[slot][e / 4][threadIdx.x];
                u[e] = f.x, u[e + 1] = f.y, u[e + 2] = f.z, u[e + 3] = f.w;
            }
            float x[kVec], d[kVec];
            piece_values(v, x);
            piece_values(w, d);
            if (s.usual) {
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) r[e] = s.usual_r(x[e], d[e]);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) r[e] = s.r(x[e], d[e]);
            }
        }
        copy(j + kDrawRing * kThreads, slot);
        slot = slot + 1 < kDrawRing ? slot + 1 : 0;
        if (best.bound == 0.0f) {  // in the whole warp
            // a first bound by each thread's largest r, and its single element
            float top = 0.0f;
            uint32_t highest = row.vocab;
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e)
                if (r[e] > top) top = r[e], highest = i + e;
            for (int k = 0; k < 2; ++k) {
                const uint32_t t = k == 0 ? lone : highest;
                if (t < row.vocab && t != s.without) best.take(s.r(t), s.u[t], t);
            }
            lone = row.vocab;
            best.share();
        }
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e)
            if (best.open(r[e], fmaxf(u[e], kUniformLo))) which |= 1u << e;
        for (; which; which &= which - 1) {
            const uint32_t t = i + __ffs(which) - 1;
            if (t < row.vocab && t != s.without) best.take(s.r(t), s.u[t], t);
        }
        best.share();
        if (base + kThreads >= end) break;
    }
    wait_copies<0>();
    return best;
}

// The largest key of the CTA, to thread 0.
__device__ __forceinline__ uint64_t cta_largest(uint64_t key, uint64_t *s_key)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(kFull, key, o);
        key = k > key ? k : key;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_key[threadIdx.x >> 5] = key;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kWarps; ++w) key = s_key[w] > key ? s_key[w] : key;
    return key;
}

// One chunk of the row at which a sequence stops; the last one writes the results.
template <class T>
__global__ void __launch_bounds__(kThreads, kDrawWave)
verify_draw_kernel(Verify a)
{
    __shared__ Part s_target[GC_MAX_DRAFTS + 1], s_draft[GC_MAX_DRAFTS + 1];
    __shared__ bool s_ok[GC_MAX_DRAFTS + 1];
    __shared__ uint64_t s_key[kWarps];
    __shared__ uint32_t s_stop, s_last;
    __shared__ int32_t s_token;
    extern __shared__ uint4 s_rings[];
    DrawRing<T> &ring = *reinterpret_cast<DrawRing<T> *>(s_rings);
    const uint32_t b = blockIdx.x / a.draws, c = blockIdx.x % a.draws;
    const float t = a.t(b), power = power_of(t);
    const bool greedy = !(t > 0.0f);
    const int32_t *ids = a.ids + size_t(b) * a.drafts;
    if (greedy && c > 0) return;
    chain_wait();
    // Where the rows' kernel has decided, only the row at which the sequence
    // stops is looked up now, the others by the CTA that writes the results.
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto target_row = [&](uint32_t j) {
        return row_part(a.x_part + (size_t(b) * (a.drafts + 1) + j) * a.chunks, a.chunks, greedy, power);
    };
    if (a.left) {
        const uint32_t j = a.drafts - a.left[b];
        if (warp == 0) {
            const Part part = target_row(j);
            if (lane == 0) s_target[j] = part, s_stop = j;
        } else if (warp == 1 && a.d && !greedy && j < a.drafts) {
            // of use only if the drafted token is one
            const Part part = row_part(a.d_part + (size_t(b) * a.drafts + j) * a.chunks, a.chunks, false, power);
            if (lane == 0) s_draft[j] = part;
        }
        __syncthreads();
    } else {
        for (uint32_t j = warp; j <= a.drafts; j += kWarps) {
            Part target, draft;
            const bool ok = decide<T>(a, b, j, target, draft);
            if (lane == 0) s_ok[j] = ok, s_target[j] = target, s_draft[j] = draft;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t j = 0;
            while (j < a.drafts && s_ok[j]) ++j;
            s_stop = j;
        }
        __syncthreads();
    }
    const uint32_t stop = s_stop;
    const T *x = static_cast<const T *>(a.x) + size_t(b) * (a.drafts + 1) * a.x_stride;
    if (greedy) {
        if (threadIdx.x == 0) {
            const uint64_t key = s_target[stop].key;
            s_token = uint32_t(key >> 32) > order_bits(-INFINITY) ? int32_t(uint32_t(~key)) : -1;
        }
    } else {
        Stop<T> s;
        const bool rejected = stop < a.drafts && a.real(uint32_t(ids[stop]));
        s.x = x + stop * a.x_stride;
        s.d = rejected && a.d ? static_cast<const T *>(a.d) + (size_t(b) * a.drafts + stop) * a.d_stride : nullptr;
        s.u = a.uniform + size_t(b) * a.u_stride;
        s.m = s_target[stop].m;
        s.inverse = s_target[stop].sum > 0.0f ? 1.0f / s_target[stop].sum : 0.0f;
        if (s.d) {
            s.dm = s_draft[stop].m;
            s.dinverse = s_draft[stop].sum > 0.0f ? 1.0f / s_draft[stop].sum : 0.0f;
        }
        s.power = power;
        s.without = rejected && !a.d ? uint32_t(ids[stop]) : ~0u;
        const Pieces<T> row(s.x, a.vocab);
        uint32_t first = min(c * a.draw, row.count), end = min(first + a.draw, row.count);
        uint64_t key;
        for (bool again = false;; again = true) {
            if (!s.d) s.dm = 0.0f, s.dinverse = 0.0f;
            s.c = s.m * power, s.dc = s.dm * power;
            s.usual = plain(s.c) && s.m < kLargest && plain(s.dc) && s.dm < kLargest;
            key = cta_largest(chunk_draw(s, row, first, end, again || c == 0, ring).key(), s_key);
            if (again) break;
            if (threadIdx.x == 0) {
                if (key) atomicMax(a.best + b, static_cast<unsigned long long>(key));
                __threadfence();
                s_last = atomicAdd(a.drawn + b, 1u) + 1 == a.draws;
                __threadfence();
            }
            __syncthreads();
            if (!s_last) return;
            key = *reinterpret_cast<volatile unsigned long long *>(a.best + b);
            if (key || s.inverse == 0.0f) break;
            // p - q rounds to nothing everywhere: p stands for it
            s.d = nullptr;
            s.without = ~0u;
            first = 0, end = row.count;
        }
        if (threadIdx.x == 0) s_token = key ? int32_t(uint32_t(~key)) : -1;
    }
    if (a.left)
        for (uint32_t j = warp; j < stop; j += kWarps) {
            const Part part = target_row(j);
            if (lane == 0) s_target[j] = part;
        }
    __syncthreads();
    if (threadIdx.x == 0) a.accepted[b] = int32_t(stop);
    for (uint32_t j = threadIdx.x; j <= a.drafts; j += kThreads) {
        const int32_t token = j < stop ? ids[j] : j == stop ? s_token : -1;
        const size_t at = size_t(b) * (a.drafts + 1) + j;
        a.tokens[at] = token;
        if (a.logprobs == nullptr) continue;
        float lp = token < 0 ? -INFINITY : 0.0f;
        if (token >= 0 && !greedy) {
            // log(w / sum) with sum = 2^k f, 1 <= f < 2: the exponent of w less k, without the roundings of either
            // (the reference may lie far from both), and log f
            const float v = sample_value(row_to_float(x[j * a.x_stride + token])), m = s_target[j].m, o = m * power;
            const int bits = __float_as_int(s_target[j].sum), k = (bits >> 23) - 127;
            const float f = __int_as_float((bits & 0x7fffff) | 0x3f800000), product = v * power;
            float z = (v - m) * power - float(k);
            if (plain(o)) z = product - o - float(k) + fmaf(v, power, -product);
            lp = fminf(z * 0.693147181f - logf(f), 0.0f);  // what is above 0 is roundings
        }
        a.logprobs[at] = lp;
    }
}

struct Plan {
    uint32_t chunk, chunks;
    bool skip;
};

Plan plan_of(size_t rows, size_t vocab, size_t elem)
{
    const size_t pieces = vocab * elem / 16 + 1, wave = gch::kSms * kWave;
    uint32_t steps = kSteps;
    while (steps > 1 && rows * gch::ceil_div(pieces, size_t(steps) * kThreads) < wave) steps /= 2;
    Plan p{steps * kThreads, uint32_t(gch::ceil_div(pieces, size_t(steps) * kThreads)), false};
    p.skip = rows * p.chunks > kSkipWaves * wave;
    return p;
}

struct Layout {
    size_t x_part, d_part, best, drawn, left, arrived, bytes;
};

Layout layout_of(size_t sequences, size_t drafts, uint32_t chunks)
{
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += gch::align_up(bytes, 256);
        return here;
    };
    l.x_part = take(sequences * (drafts + 1) * chunks * sizeof(Part));
    l.d_part = take(sequences * drafts * chunks * sizeof(Part));
    l.best = take(sequences * 8);  // from here on: zeros where chunks decide
    l.drawn = take(sequences * 4);
    l.left = take(sequences * 4);
    l.arrived = take(sequences * drafts * 4);
    l.bytes = at;
    return l;
}

template <class T>
cudaError_t run_verify(Verify a, uint8_t *ws, cudaStream_t s)
{
    const size_t target_rows = size_t(a.sequences) * (a.drafts + 1), draft_rows = a.d ? size_t(a.sequences) * a.drafts : 0;
    const Plan plan = plan_of(target_rows + draft_rows, a.vocab, sizeof(T));
    const Layout l = layout_of(a.sequences, a.drafts, plan.chunks);
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.x_part = reinterpret_cast<Part *>(ws + l.x_part);
    a.d_part = reinterpret_cast<Part *>(ws + l.d_part);
    a.best = reinterpret_cast<unsigned long long *>(ws + l.best);
    a.drawn = reinterpret_cast<uint32_t *>(ws + l.drawn);
    if (plan.skip && a.drafts > 0) {
        a.left = reinterpret_cast<uint32_t *>(ws + l.left);
        a.arrived = reinterpret_cast<uint32_t *>(ws + l.arrived);
        const cudaError_t e = cudaMemsetAsync(ws + l.best, 0, l.bytes - l.best, s);
        if (e != cudaSuccess) return e;
    }
    // The draw's chunks: as many CTAs as run at a time, a piece to a thread at least.
    const uint32_t pieces = uint32_t(size_t(a.vocab) * sizeof(T) / 16 + 1);
    const uint32_t most = uint32_t(gch::ceil_div(pieces, size_t(kThreads)));
    a.draws = uint32_t(gch::kSms * kDrawWave / a.sequences);
    a.draws = a.draws < 1 ? 1 : a.draws < most ? a.draws : most;
    a.draw = uint32_t(gch::ceil_div(pieces, a.draws));
    const dim3 grid(a.sequences * (a.d ? 2 : 1), plan.chunks, a.drafts + 1);
    verify_rows_kernel<T><<<grid, kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the attribute lasts as long as the process: set once for each device
    constexpr size_t kSmem = sizeof(DrawRing<T>);
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    e = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (e == cudaSuccess && (dev > 63 || !(set.load(std::memory_order_relaxed) & bit))) {
        e = cudaFuncSetAttribute(verify_draw_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
        if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
    return gch::launch_next(verify_draw_kernel<T>, dim3(a.sequences * a.draws), dim3(kThreads), kSmem, s, a);
}

}  // namespace

namespace gch {

size_t sample_verify_workspace_bytes(size_t sequences, size_t drafts, size_t vocab)
{
    // the most chunks of any type, with a draft's rows or without
    uint32_t chunks = 1;
    for (size_t elem : {size_t(2), size_t(4)})
        for (size_t rows : {sequences * (drafts + 1), sequences * (2 * drafts + 1)}) {
            const uint32_t c = plan_of(rows, vocab, elem).chunks;
            chunks = c > chunks ? c : chunks;
            if (rows * c > GC_MAX_ELEMENTS) return 0;  // CTAs of one launch
        }
    return layout_of(sequences, drafts, chunks).bytes + 256;
}

cudaError_t launch_sample_verify(const void *logits, size_t logits_stride, const void *draft_logits,
                                 size_t draft_stride, uint32_t sequences, uint32_t drafts, uint32_t vocab,
                                 gc_row_dtype dt, const int32_t *ids, const float *accept, const float *uniform,
                                 size_t uniform_stride, const float *temperature, int32_t *tokens, int32_t *accepted,
                                 float *logprobs, uint8_t *ws, cudaStream_t s)
{
    Verify a{};
    a.sequences = sequences, a.drafts = drafts, a.vocab = vocab;
    a.x_stride = logits_stride, a.d_stride = draft_stride, a.u_stride = uniform_stride;
    a.x = logits, a.d = draft_logits, a.ids = ids;
    a.accept = accept, a.uniform = uniform, a.temperature = temperature;
    a.tokens = tokens, a.accepted = accepted, a.logprobs = logprobs;
    if (dt == GC_ROW_F32) return run_verify<float>(a, ws, s);
    if (dt == GC_ROW_BF16) return run_verify<__nv_bfloat16>(a, ws, s);
    return run_verify<__half>(a, ws, s);
}

}  // namespace gch
