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
// then by sequence: where there are more than the GPU holds at a time, the
// last chunk of a position decides it, and chunks of later positions of a
// sequence that has stopped are not read.
#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;             // pieces of 16 bytes that a thread has under way
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLargest = 3.402823466e38f;
constexpr float kUniformLo = 0x1p-25f, kUniformHi = 1.0f - 0x1p-24f;

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
    uint32_t *stop, *arrived;   // per sequence: first rejected position; per position: chunks done; NULL: not kept

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

__device__ __forceinline__ float batch_weight(float x, float m, float power)
{
    // NaN weighs nothing, +inf as much as the largest value
    return pow2(fminf(fmaxf((sample_value(x) - m) * power, -INFINITY), 0.0f));
}

// m and sum joined with another maximum and sum.
__device__ __forceinline__ void join(float &m, float &sum, float m2, float sum2, float power)
{
    const float top = fmaxf(m, m2);
    if (top > -INFINITY) {
        sum = sum * pow2((m - top) * power) + sum2 * pow2((m2 - top) * power);
        m = top;
    }
}

// A chunk's maximum and sum, to lane 0 of warp 0.
template <class T>
__device__ __forceinline__ Part chunk_sum(const Pieces<T> &row, uint32_t first, uint32_t end, bool singles, float power,
                                          Part *s_part)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    float m = -INFINITY, sum = 0.0f;
    if (singles) {
        const uint32_t i = row.single(threadIdx.x);
        if (i < row.vocab) {
            m = sample_value(row_to_float(row.x[i]));
            sum = m > -INFINITY ? 1.0f : 0.0f;
        }
    }
    for (uint32_t base = first + threadIdx.x; base < end; base += kBatch * kThreads) {
        Piece<T, kVec> v[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const uint32_t j = base + q * kThreads;
            if (j < end) {
                v[q] = load_piece<T, kVec>(row.x + row.head + size_t(j) * kVec);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) v[q].v[e] = row_from_float<T>(-INFINITY);
            }
        }
        float top = m;
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) top = fmaxf(top, row_to_float(v[q].v[e]));
        top = fminf(top, kLargest);
        if (!(top > -INFINITY)) continue;
        float more = 0.0f;
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) more += pow2((row_to_float(v[q].v[e]) - top) * power);
        if (!(more <= float(kBatch * kVec))) {  // a NaN or an infinity
            more = 0.0f;
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
#pragma unroll
                for (uint32_t e = 0; e < kVec; ++e) more += batch_weight(row_to_float(v[q].v[e]), top, power);
        }
        sum = (m > -INFINITY ? sum * pow2((m - top) * power) : 0.0f) + more;
        m = top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) join(m, sum, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, sum, o), power);
    Part p;
    p.m = m, p.sum = sum;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = p;
    __syncthreads();
    if (threadIdx.x < kWarps) {
        m = s_part[threadIdx.x].m, sum = s_part[threadIdx.x].sum;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
            join(m, sum, __shfl_xor_sync(0xffu, m, o), __shfl_xor_sync(0xffu, sum, o), power);
        p.m = m, p.sum = sum;
    }
    return p;
}

// The key of the first of a chunk's largest values, to lane 0 of warp 0.
template <class T>
__device__ __forceinline__ Part chunk_first(const Pieces<T> &row, uint32_t first, uint32_t end, bool singles,
                                            Part *s_part)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    uint64_t key = first_key(-INFINITY, ~0u);
    if (singles) {
        const uint32_t i = row.single(threadIdx.x);
        if (i < row.vocab) key = first_key(sample_value(row_to_float(row.x[i])), i);
    }
    for (uint32_t base = first + threadIdx.x; base < end; base += kBatch * kThreads) {
        Piece<T, kVec> v[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const uint32_t j = base + q * kThreads;
            if (j < end) v[q] = load_piece<T, kVec>(row.x + row.head + size_t(j) * kVec);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const uint32_t j = base + q * kThreads;
            if (j >= end) continue;
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) {
                const uint64_t k = first_key(sample_value(row_to_float(v[q].v[e])), row.head + j * kVec + e);
                key = k > key ? k : key;
            }
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) join(m, sum, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, sum, o), power);
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
    const double wp = batch_weight(row_to_float(x[id]), target.m, power);
    double wq = 1.0;
    if (a.d) {
        draft = row_part(a.d_part + at * a.chunks, a.chunks, false, power);
        const T *d = static_cast<const T *>(a.d) + at * a.d_stride;
        wq = draft.sum > 0.0f ? batch_weight(row_to_float(d[id]), draft.m, power) : 0.0f;
    }
    const double u = fminf(fmaxf(a.accept[at], kUniformLo), kUniformHi);
    return target.sum > 0.0f && u * wq * double(target.sum) < wp * (draft.sum > 0.0f ? double(draft.sum) : 1.0);
}

// One chunk of one row.
template <class T>
__global__ void __launch_bounds__(kThreads)
verify_rows_kernel(Verify a)
{
    __shared__ Part s_part[kWarps];
    chain_start();
    // unit -> position, sequence, target or draft, chunk
    const uint32_t kinds = a.d ? 2 : 1, each = a.sequences * kinds * a.chunks;
    uint32_t unit = blockIdx.x, j = unit / each, kind = 0;
    if (j >= a.drafts) j = a.drafts;
    unit -= j * each;
    const uint32_t c = unit % a.chunks;
    unit /= a.chunks;
    if (j < a.drafts) {
        kind = unit % kinds;
        unit /= kinds;
    }
    const uint32_t b = unit;
    if (a.stop && *reinterpret_cast<volatile uint32_t *>(a.stop + b) < j) return;
    if (j == 0 && kind == 0 && c == 0 && threadIdx.x == 0) {
        a.best[b] = 0;
        a.drawn[b] = 0;
    }
    const float t = a.t(b), power = power_of(t);
    const bool greedy = !(t > 0.0f);
    if (kind == 1 && greedy) return;
    // a position past the first drafted token that is none is not reached
    const int32_t *ids = a.ids + size_t(b) * a.drafts;
    for (uint32_t i = 0; i < j + kind; ++i)
        if (!a.real(uint32_t(ids[i]))) return;

    const T *x = kind == 0 ? static_cast<const T *>(a.x) + (size_t(b) * (a.drafts + 1) + j) * a.x_stride
                           : static_cast<const T *>(a.d) + (size_t(b) * a.drafts + j) * a.d_stride;
    const Pieces<T> row(x, a.vocab);
    const uint32_t first = min(c * a.chunk, row.count), end = min(first + a.chunk, row.count);
    const Part p = greedy ? chunk_first(row, first, end, c == 0, s_part)
                          : chunk_sum(row, first, end, c == 0, power, s_part);
    Part *to = kind == 0 ? a.x_part + (size_t(b) * (a.drafts + 1) + j) * a.chunks + c
                         : a.d_part + (size_t(b) * a.drafts + j) * a.chunks + c;
    if (threadIdx.x == 0) to->key = p.key;
    if (a.stop == nullptr || j == a.drafts || threadIdx.x >= 32) return;
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        before = atomicAdd(a.arrived + size_t(b) * a.drafts + j, 1u);
        __threadfence();
    }
    before = __shfl_sync(kFull, before, 0);
    const bool none = !a.real(uint32_t(ids[j]));  // then the draft's row is not read
    if (before + 1 != a.chunks * (greedy || none ? 1 : kinds)) return;
    Part target, draft;
    if (!decide<T>(a, b, j, target, draft) && threadIdx.x == 0) atomicMin(a.stop + b, j);
}

// Of the tokens offered, the largest r / -log v; equal ones, the lowest index.
struct Best {
    float ratio = 0.0f;
    uint32_t index = ~0u;
    __device__ __forceinline__ void take(float r, float v, uint32_t i)
    {
        const float q = r / -logf(fminf(fmaxf(v, kUniformLo), kUniformHi));
        if (q > ratio || (q == ratio && i < index)) {
            ratio = q;
            index = i;
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
    float m, inverse, dm, dinverse, power;
    uint32_t without;   // a token that cannot be drawn

    __device__ __forceinline__ float p(float v) const { return batch_weight(v, m, power) * inverse; }
    __device__ __forceinline__ float q(float v) const { return batch_weight(v, dm, power) * dinverse; }
    __device__ __forceinline__ float r(uint32_t i) const
    {
        float w = p(row_to_float(x[i]));
        if (d) w = fmaxf(w - q(row_to_float(d[i])), 0.0f);
        return i == without ? 0.0f : w;
    }
};

template <class T>
__device__ __forceinline__ Best chunk_draw(const Stop<T> &s, const Pieces<T> &row, uint32_t first, uint32_t end,
                                           bool singles)
{
    constexpr uint32_t kVec = Pieces<T>::kVec;
    Best best;
    if (singles) {
        const uint32_t i = row.single(threadIdx.x);
        if (i < row.vocab) best.take(s.r(i), s.u[i], i);
    }
    const bool d_whole = s.d && ((reinterpret_cast<uintptr_t>(s.d + row.head)) & 15u) == 0;
    const bool u_whole = ((reinterpret_cast<uintptr_t>(s.u + row.head)) & 15u) == 0;
    for (uint32_t base = first; base < end; base += kThreads) {
        const uint32_t j = base + threadIdx.x;
        if (j >= end) break;
        const uint32_t i = row.head + j * kVec;
        const Piece<T, kVec> v = load_piece<T, kVec>(row.x + i);
        Piece<T, kVec> w;
        float u[kVec];
        if (d_whole) {
            w = load_piece<T, kVec>(s.d + i);
        } else if (s.d) {
#pragma unroll
            for (uint32_t e = 0; e < kVec; ++e) w.v[e] = s.d[i + e];
        }
#pragma unroll
        for (uint32_t e = 0; e < kVec; e += 4) {
            if (u_whole) {
                const float4 f = __ldcs(reinterpret_cast<const float4 *>(s.u + i + e));
                u[e] = f.x, u[e + 1] = f.y, u[e + 2] = f.z, u[e + 3] = f.w;
            } else {
#pragma unroll
                for (uint32_t k = e; k < e + 4; ++k) u[k] = __ldcs(s.u + i + k);
            }
        }
#pragma unroll
        for (uint32_t e = 0; e < kVec; ++e) {
            float r = s.p(row_to_float(v.v[e]));
            if (s.d) r = fmaxf(r - s.q(row_to_float(w.v[e])), 0.0f);
            if (r > 0.0f && i + e != s.without) best.take(r, u[e], i + e);
        }
    }
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
__global__ void __launch_bounds__(kThreads)
verify_draw_kernel(Verify a)
{
    __shared__ Part s_target[GC_MAX_DRAFTS + 1], s_draft[GC_MAX_DRAFTS + 1];
    __shared__ bool s_ok[GC_MAX_DRAFTS + 1];
    __shared__ uint64_t s_key[kWarps];
    __shared__ uint32_t s_stop, s_last;
    __shared__ int32_t s_token;
    const uint32_t b = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    const float t = a.t(b), power = power_of(t);
    const bool greedy = !(t > 0.0f);
    const int32_t *ids = a.ids + size_t(b) * a.drafts;
    if (greedy && c > 0) return;
    chain_wait();
    for (uint32_t j = threadIdx.x >> 5; j <= a.drafts; j += kWarps) {
        Part target, draft;
        const bool ok = decide<T>(a, b, j, target, draft);
        if ((threadIdx.x & 31) == 0) {
            s_ok[j] = ok;
            s_target[j] = target;
            s_draft[j] = draft;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t j = 0;
        while (j < a.drafts && s_ok[j]) ++j;
        s_stop = j;
    }
    __syncthreads();
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
        s.dm = s_draft[stop].m;
        s.dinverse = s_draft[stop].sum > 0.0f ? 1.0f / s_draft[stop].sum : 0.0f;
        s.power = power;
        s.without = rejected && !a.d ? uint32_t(ids[stop]) : ~0u;
        const Pieces<T> row(s.x, a.vocab);
        const uint32_t first = min(c * a.chunk, row.count), end = min(first + a.chunk, row.count);
        uint64_t key = cta_largest(chunk_draw(s, row, first, end, c == 0).key(), s_key);
        if (threadIdx.x == 0) {
            if (key) atomicMax(a.best + b, static_cast<unsigned long long>(key));
            __threadfence();
            s_last = atomicAdd(a.drawn + b, 1u) + 1 == a.chunks;
            __threadfence();
        }
        __syncthreads();
        if (!s_last) return;
        key = *reinterpret_cast<volatile unsigned long long *>(a.best + b);
        if (key == 0 && s.inverse > 0.0f) {
            // p - q rounds to nothing everywhere: p stands for it
            s.d = nullptr;
            s.without = ~0u;
            key = cta_largest(chunk_draw(s, row, 0, row.count, true).key(), s_key);
        }
        if (threadIdx.x == 0) s_token = key ? int32_t(uint32_t(~key)) : -1;
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
            const float z = (sample_value(row_to_float(x[j * a.x_stride + token])) - s_target[j].m) / t;
            lp = z - logf(s_target[j].sum);
        }
        a.logprobs[at] = lp;
    }
}

// Chunks: eight pieces per thread, 32 KB, where that makes more CTAs than the
// GPU holds, else fewer.
constexpr uint32_t kSteps = 8, kWave = 8;  // kWave: CTAs per SM

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
    p.skip = rows * p.chunks > wave;
    return p;
}

struct Layout {
    size_t x_part, d_part, best, drawn, stop, arrived, bytes;
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
    l.best = take(sequences * 8);
    l.drawn = take(sequences * 4);
    l.stop = take(sequences * 4);
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
        a.stop = reinterpret_cast<uint32_t *>(ws + l.stop);
        a.arrived = reinterpret_cast<uint32_t *>(ws + l.arrived);
        cudaError_t e = cudaMemsetAsync(a.stop, 0xff, size_t(a.sequences) * 4, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(a.arrived, 0, size_t(a.sequences) * a.drafts * 4, s);
        if (e != cudaSuccess) return e;
    }
    verify_rows_kernel<T><<<uint32_t((target_rows + draft_rows) * plan.chunks), kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return gch::launch_next(verify_draw_kernel<T>, dim3(a.sequences * plan.chunks), dim3(kThreads), 0, s, a);
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
