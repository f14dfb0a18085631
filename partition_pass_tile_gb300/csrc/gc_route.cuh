// gc_route.cuh -- what the routing kernels (route.cu, route_grad.cu) share: how
// a token's logits lie in the lanes of a warp or of a part of one, and their
// weights.
#pragma once

#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace gcd {

constexpr uint32_t kRouteFull = 0xffffffffu;
constexpr uint32_t kRouteNone = 0x007fffffu;  // order_bits(-inf): no expert
constexpr float kLog2e = 1.44269504f;

// Up to kSmallExperts experts a token belongs to a group of 1, 2 or 4 lanes with
// eight each, more of them to a warp with V each: 131072 tokens of 32 experts,
// top-4, take GROUP us by groups and WARP by warps, of 64 GROUP64 and WARP64.
constexpr uint32_t kSmallExperts = 32;
constexpr int kGroupValues = 8;

inline uint32_t route_lanes(uint32_t experts)
{
    if (experts > kSmallExperts) return 32;
    uint32_t lanes = 1;
    while (lanes * kGroupValues < experts) lanes *= 2;
    return lanes;
}

// Experts of a lane of a warp.
inline int route_values(uint32_t experts)
{
    for (int v : {2, 4, 8, 16})
        if (experts <= 32u * uint32_t(v)) return v;
    return 64;
}

// This lane's logits of a token, -inf where there is none.
template <class T, int N, int V>
struct Logits {
    Piece<T, N> p[V / N];

    __device__ __forceinline__ void load(const T *__restrict__ row, uint32_t first, uint32_t experts, bool live)
    {
#pragma unroll
        for (int i = 0; i < V / N; ++i) {
            if (live && first + i * N < experts) {
                p[i] = load_piece<T, N>(row + first + i * N);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) p[i].v[e] = row_from_float<T>(-INFINITY);
            }
        }
    }
    __device__ __forceinline__ float operator[](int v) const { return row_to_float(p[v / N].v[v % N]); }
    __device__ __forceinline__ void values(float (&x)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V / N; ++i) {
            float y[N];
            piece_values(p[i], y);
#pragma unroll
            for (int e = 0; e < N; ++e) x[i * N + e] = y[e];
        }
    }
};

// exp(x - m) as a power of two.  c = m log2(e) is taken off by a multiply-add,
// whose only rounding is the exponent's (every weight of a token carries the
// same 2^(m log2(e) - c)), unless the logits are not all finite and small.
struct Exponent {
    float m, c;
    bool usual;
    __device__ __forceinline__ float weight(float x) const
    {
        return pow2(usual ? fmaf(x, kLog2e, -c) : (sample_value(x) - m) * kLog2e);
    }
};

// The sum over a warp.
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kRouteFull, v, o);
    return v;
}

// A warp's token: w[V] are the weights exp(x - m) of its logits x[V]; returns
// their sum, 0 if no expert is open, and the order bits of the largest logit of
// the warp (top) and of the lane (best).  Logits that are not all finite and
// small leave cleaned.
template <int V>
__device__ __forceinline__ float warp_weights(float (&x)[V], float (&w)[V], Exponent &exponent, uint32_t &top,
                                              uint32_t &best)
{
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) most = fmaxf(most, x[v]);
    best = order_bits(most);
    top = __reduce_max_sync(kRouteFull, best);
    exponent.m = order_value(top);
    exponent.c = exponent.m * kLog2e;
    exponent.usual = true;
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = pow2(fmaf(x[v], kLog2e, -exponent.c));
        total += w[v];
    }
    total = warp_sum(total);
    if (total <= 1.5f * 32 * V && fabsf(exponent.c) < 0x1p100f) return total;
    // no expert, a NaN, an infinity or a very large logit
    exponent.usual = false;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = sample_value(x[v]);
    best = order_bits(fminf(most, 3.402823466e38f));
    top = __reduce_max_sync(kRouteFull, best);
    exponent.m = top > kRouteNone ? order_value(top) : 0.0f;
    total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = exponent.weight(x[v]);
        total += w[v];
    }
    return warp_sum(total);
}

// 1 / x of a sum of weights, off by at most 2^-23 of itself.
__device__ __forceinline__ float inverse_of(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The sums over a CTA of W warps, of whole numbers and of floats; every thread
// calls them and has the result.
template <int W>
__device__ __forceinline__ uint32_t cta_count(uint32_t v, uint32_t *s_warp)
{
    v = __reduce_add_sync(kRouteFull, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(kRouteFull, (threadIdx.x & 31) < W ? s_warp[threadIdx.x & 31] : 0u);
}

template <int W>
__device__ __forceinline__ float cta_sum(float v, uint32_t *s_warp)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = __float_as_uint(v);
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < W ? __uint_as_float(s_warp[threadIdx.x & 31]) : 0.0f);
}

// A group of 1, 2 or 4 lanes.
struct Group {
    uint32_t lanes, lane, mask;
    __device__ __forceinline__ explicit Group(uint32_t lanes_) : lanes(lanes_), lane(threadIdx.x & (lanes_ - 1))
    {
        mask = ((1u << lanes) - 1u) << ((threadIdx.x & 31) - lane);
    }
    __device__ __forceinline__ uint32_t largest(uint32_t v) const
    {
        for (uint32_t o = lanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kRouteFull, v, o));
        return v;
    }
    __device__ __forceinline__ float sum(float v) const
    {
        for (uint32_t o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kRouteFull, v, o);
        return v;
    }
};

struct Pick {
    float x;
    int32_t id;
};

// Pieces of 16 bytes (or of a lane's share) where pointers, strides and experts
// allow it, else elements.  CALL(T, N) for groups, CALL_WARP(T, N, V) for warps.
#define GC_ROUTE_BY_VALUES(T, values, whole, CALL_WARP)                                             \
    switch (values) {                                                                               \
    case 2: if (whole) { return CALL_WARP(T, 2, 2); } return CALL_WARP(T, 1, 2);                    \
    case 4: if (whole) { return CALL_WARP(T, 4, 4); } return CALL_WARP(T, 1, 4);                    \
    case 8: if (whole) { return CALL_WARP(T, int(16 / sizeof(T)), 8); } return CALL_WARP(T, 1, 8);  \
    case 16: if (whole) { return CALL_WARP(T, int(16 / sizeof(T)), 16); } return CALL_WARP(T, 1, 16); \
    default: if (whole) { return CALL_WARP(T, int(16 / sizeof(T)), 64); } return CALL_WARP(T, 1, 64); \
    }
#define GC_ROUTE_BY_SIZE(T, experts, whole, CALL, CALL_WARP)                        \
    if (experts > kSmallExperts) { GC_ROUTE_BY_VALUES(T, route_values(experts), whole, CALL_WARP) } \
    if (whole) { return CALL(T, int(16 / sizeof(T))); }                             \
    return CALL(T, 1);
#define GC_ROUTE_BY_DTYPE(dt, experts, whole, CALL, CALL_WARP)                                  \
    if (dt == GC_ROW_F32) { GC_ROUTE_BY_SIZE(float, experts, whole, CALL, CALL_WARP) }          \
    if (dt == GC_ROW_BF16) { GC_ROUTE_BY_SIZE(__nv_bfloat16, experts, whole, CALL, CALL_WARP) } \
    GC_ROUTE_BY_SIZE(__half, experts, whole, CALL, CALL_WARP)

}  // namespace gcd
