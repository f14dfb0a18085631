// sample.cu -- one token per row of logits from given uniform random numbers
// (gc_sample): temperature, top-k, top-p, min-p, then the Gumbel-max draw.
//
// Every filter keeps a prefix of one order, x descending and equal values by
// index, which is the descending order of the 64-bit key
//     (order-preserving bits of x) << 32 | ~index.
// Top-k and top-p are each one cut of that key, found by radix selection: a
// histogram of the next 8 bits of the tokens that share the cut's bits so
// far, with the tokens counted (top-k) or their weights added (top-p).  The
// weights are added as whole multiples of 2^-40 of the largest weight, so
// the sum does not depend on the order of the atomics.
#include "gc_internal.h"
#include "gc_rows.cuh"

namespace {

using namespace gcd;

constexpr int kSampleThreads = 1024;
constexpr int kSampleWarps = kSampleThreads / 32;
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

__device__ __forceinline__ float scaled(float x, float m, float t)
{
    const float d = x - m;
    return d == -INFINITY ? d : d / t;
}

struct SampleSmem {
    uint64_t warp[kSampleWarps];
    uint64_t hist[256];
    uint64_t cut, above;
    double mass[kSampleWarps];
    bool found;
};

template <class V, class Op>
__device__ __forceinline__ V block_reduce(V v, V *s_warp, Op op)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    V r = s_warp[0];
    for (int w = 1; w < kSampleWarps; ++w) r = op(r, s_warp[w]);
    return r;
}

// The largest key K such that the amounts of all keys >= K sum to at least
// target (>= 1); 0 if they all together do not.  amount(i, key) of token i;
// `each` calls its argument for every token with its key.
template <class Each>
__device__ __forceinline__ uint64_t select_cut(uint64_t target, SampleSmem &sm, const Each &each)
{
    uint64_t prefix = 0u, above = 0u;
    for (int shift = 56; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int b = threadIdx.x; b < 256; b += kSampleThreads) sm.hist[b] = 0u;
        if (threadIdx.x == 0) sm.found = false;
        __syncthreads();
        each([&](uint64_t key, uint64_t amount) {
            if (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(reinterpret_cast<unsigned long long *>(&sm.hist[(key >> shift) & 255u]),
                          static_cast<unsigned long long>(amount));
        });
        __syncthreads();
        if (threadIdx.x < 32) {
            // Lane l owns bins 255 - 8 l down to 248 - 8 l.
            const int top = 255 - 8 * int(threadIdx.x);
            uint64_t sum = 0u;
            for (int k = 0; k < 8; ++k) sum += sm.hist[top - k];
            uint64_t incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (int(threadIdx.x) >= o) incl += y;
            }
            uint64_t before = above + incl - sum;
            if (before < target && before + sum >= target) {
                for (int k = 0; k < 8; ++k) {
                    const uint64_t h = sm.hist[top - k];
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

template <class T>
__global__ void __launch_bounds__(kSampleThreads)
sample_kernel(const T *__restrict__ logits, size_t logits_stride, uint32_t vocab,
              const float *__restrict__ uniform, size_t uniform_stride, const float *__restrict__ temperature,
              const int32_t *__restrict__ top_k, const float *__restrict__ top_p, const float *__restrict__ min_p,
              int32_t *__restrict__ tokens, float *__restrict__ logprobs)
{
    __shared__ SampleSmem sm;
    const uint32_t row = blockIdx.x;
    const T *x = logits + size_t(row) * logits_stride;
    const float *u = uniform + size_t(row) * uniform_stride;
    auto value = [&](uint32_t i) { return sample_value(row_to_float(x[i])); };
    auto larger = [](auto a, auto b) { return a > b ? a : b; };

    // The first of the order.
    uint64_t best = 0u;
    for (uint32_t i = threadIdx.x; i < vocab; i += kSampleThreads) {
        const float v = value(i);
        if (v > -INFINITY) best = larger(best, order_key(v, i));
    }
    best = block_reduce(best, sm.warp, larger);
    const float t = temperature ? temperature[row] : 1.0f;
    if (best == 0u || uniform == nullptr || !(t > 0.0f)) {
        if (threadIdx.x == 0) {
            tokens[row] = best == 0u ? -1 : int32_t(~uint32_t(best));
            if (logprobs) logprobs[row] = best == 0u ? -INFINITY : 0.0f;
        }
        return;
    }
    const float m = value(~uint32_t(best));

    uint64_t cut = 0u;
    const int32_t k = top_k ? top_k[row] : 0;
    if (k > 0 && uint32_t(k) < vocab)
        cut = select_cut(uint64_t(k), sm, [&](auto add) {
            for (uint32_t i = threadIdx.x; i < vocab; i += kSampleThreads) {
                const float v = value(i);
                if (v > -INFINITY) add(order_key(v, i), 1u);
            }
        });
    const float p = top_p ? top_p[row] : 1.0f;
    if (p < 1.0f) {
        auto fixed = [&](auto add) {
            for (uint32_t i = threadIdx.x; i < vocab; i += kSampleThreads) {
                const float v = value(i);
                const uint64_t key = order_key(v, i);
                if (v > -INFINITY && key >= cut)
                    add(key, uint64_t(__float2ull_rn(expf(scaled(v, m, t)) * kFixed)));
            }
        };
        uint64_t sum = 0u;
        fixed([&](uint64_t, uint64_t w) { sum += w; });
        sum = block_reduce(sum, sm.warp, [](uint64_t a, uint64_t b) { return a + b; });
        const double target = ceil(double(fmaxf(p, 0.0f)) * double(sum));
        const uint64_t cut_p = select_cut(target < 1.0 ? 1u : uint64_t(target), sm, fixed);
        cut = larger(cut, cut_p);
    }
    const float q0 = min_p ? min_p[row] : 0.0f;
    const float q = q0 > 0.0f ? fminf(q0, 1.0f) : 0.0f;

    // What is kept: its weight, and the draw.
    float sum = 0.0f;
    best = 0u;
    for (uint32_t i = threadIdx.x; i < vocab; i += kSampleThreads) {
        const float v = value(i);
        if (!(v > -INFINITY) || order_key(v, i) < cut) continue;
        const float z = scaled(v, m, t), w = expf(z);
        if (w < q || w == 0.0f) continue;
        sum += w;
        if (z < -20.0f) continue;
        const float r = fminf(fmaxf(u[i], kUniformLo), kUniformHi);
        best = larger(best, order_key(z - logf(-logf(r)), i));
    }
    best = block_reduce(best, sm.warp, larger);
    const double mass = block_reduce(double(sum), sm.mass, [](double a, double b) { return a + b; });
    if (threadIdx.x == 0) {
        const uint32_t i = ~uint32_t(best);
        tokens[row] = int32_t(i);
        if (logprobs) logprobs[row] = scaled(value(i), m, t) - logf(float(mass));
    }
}

template <class T>
void run_sample(const void *logits, size_t logits_stride, uint32_t rows, uint32_t vocab, const float *uniform,
                size_t uniform_stride, const float *temperature, const int32_t *top_k, const float *top_p,
                const float *min_p, int32_t *tokens, float *logprobs, cudaStream_t s)
{
    sample_kernel<T><<<rows, kSampleThreads, 0, s>>>(static_cast<const T *>(logits), logits_stride, vocab, uniform,
                                                     uniform_stride, temperature, top_k, top_p, min_p, tokens,
                                                     logprobs);
}

}  // namespace

namespace gch {

cudaError_t launch_sample(const void *logits, size_t logits_stride, uint32_t rows, uint32_t vocab, gc_row_dtype dt,
                          const float *uniform, size_t uniform_stride, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                          float *logprobs, cudaStream_t s)
{
#define GC_SAMPLE_CALL(T) run_sample<T>(logits, logits_stride, rows, vocab, uniform, uniform_stride, temperature, \
                                        top_k, top_p, min_p, tokens, logprobs, s)
    if (dt == GC_ROW_F32) GC_SAMPLE_CALL(float);
    else if (dt == GC_ROW_BF16) GC_SAMPLE_CALL(__nv_bfloat16);
    else GC_SAMPLE_CALL(__half);
    return cudaGetLastError();
}

}  // namespace gch
