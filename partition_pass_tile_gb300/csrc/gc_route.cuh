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
// eight each, more of them to a team of 16 or 32 lanes: 131072 tokens of 32
// float32, top-4, take 26 us by groups and their gradient 12, by warps 55 and 58.
constexpr uint32_t kSmallExperts = 32;
constexpr int kGroupValues = 8;

inline uint32_t route_lanes(uint32_t experts)
{
    uint32_t lanes = 1;
    while (lanes * kGroupValues < experts) lanes *= 2;
    return lanes;
}

// This lane's logits of a token, -inf where there is none: pieces of N, each G
// pieces behind the one before, so that the G lanes of a team read side by side
// (G = 1: a lane's experts are neighbours).
template <class T, int N, int V, int G>
struct Logits {
    Piece<T, N> p[V / N];

    // The expert of a lane's element v.
    static __device__ __forceinline__ uint32_t expert(uint32_t first, int v)
    {
        return first + uint32_t(v / N * (G * N) + v % N);
    }
    __device__ __forceinline__ void load(const T *__restrict__ row, uint32_t first, uint32_t experts, bool live)
    {
#pragma unroll
        for (int i = 0; i < V / N; ++i) {
            if (live && first + i * G * N < experts) {
                p[i] = load_piece<T, N>(row + first + i * G * N);
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
// same 2^(m log2(e) - c), near 1), unless the logits are not all finite or large.
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

// A team of G lanes; all lanes of the warp call these together.
template <int G>
__device__ __forceinline__ float team_sum(float v)
{
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kRouteFull, v, o);
    return v;
}

template <int G>
__device__ __forceinline__ uint32_t team_max(uint32_t v)
{
    if constexpr (G == 32) {
        return __reduce_max_sync(kRouteFull, v);
    } else {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kRouteFull, v, o));
        return v;
    }
}

template <int G>
__device__ __forceinline__ uint32_t team_ballot(bool p)
{
    const uint32_t b = __ballot_sync(kRouteFull, p);
    if constexpr (G == 32) return b;
    else return (b >> (threadIdx.x & 31 & ~(G - 1))) & ((1u << G) - 1u);
}

// A team's token: w[V] are the weights exp(x - m) of its logits x[V]; returns
// their sum, 0 if no expert is open, and the order bits of the largest logit of
// the team (top) and of the lane (best).  Logits that are not all finite and
// small leave cleaned.
template <int G, int V>
__device__ __forceinline__ float team_weights(float (&x)[V], float (&w)[V], Exponent &exponent, uint32_t &top,
                                              uint32_t &best)
{
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) most = fmaxf(most, x[v]);
    best = order_bits(most);
    top = team_max<G>(best);
    exponent.m = order_value(top);
    exponent.c = exponent.m * kLog2e;
    exponent.usual = true;
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = pow2(fmaf(x[v], kLog2e, -exponent.c));
        total += w[v];
    }
    total = team_sum<G>(total);
    const bool odd = !(total <= 1.5f * G * V && fabsf(exponent.c) < 0x1p24f);
    if (!__any_sync(kRouteFull, odd)) return total;
    // a team without an expert, or with a NaN, an infinity or a very large logit: the others keep what they have
    const uint32_t clean_best = order_bits(fminf(most, 3.402823466e38f)), clean_top = team_max<G>(clean_best);
    float again = 0.0f;
    if (odd) {
        best = clean_best, top = clean_top;
        exponent.usual = false;
        exponent.m = top > kRouteNone ? order_value(top) : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = sample_value(x[v]);
            w[v] = exponent.weight(x[v]);
            again += w[v];
        }
    }
    again = team_sum<G>(again);
    return odd ? again : total;
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
// allow it, else elements.  CALL(T, N) for groups, CALL_TEAM(T, N, V, G) for
// teams: 16 lanes up to 256 experts, else the whole warp.  WARP(T, whole): what
// comes before the teams of 16 lanes; GC_ROUTE_NO_WARP where they do always.
#define GC_ROUTE_TEAM(T, whole, V, G, CALL_TEAM)                                            \
    {                                                                                       \
        constexpr int kMost = 16 / int(sizeof(T)), kPiece = V < kMost ? V : kMost;          \
        if (whole) return CALL_TEAM(T, kPiece, V, G);                                       \
        return CALL_TEAM(T, 1, V, G);                                                       \
    }
#define GC_ROUTE_NO_WARP(T, whole)
#define GC_ROUTE_BY_SIZE(T, experts, whole, CALL, CALL_TEAM, WARP)                          \
    if (experts <= kSmallExperts) {                                                         \
        if (whole) return CALL(T, int(16 / sizeof(T)));                                     \
        return CALL(T, 1);                                                                  \
    }                                                                                       \
    WARP(T, whole)                                                                          \
    if (experts <= 64) GC_ROUTE_TEAM(T, whole, 4, 16, CALL_TEAM)                            \
    if (experts <= 128) GC_ROUTE_TEAM(T, whole, 8, 16, CALL_TEAM)                           \
    if (experts <= 256) GC_ROUTE_TEAM(T, whole, 16, 16, CALL_TEAM)                          \
    if (experts <= 512) GC_ROUTE_TEAM(T, whole, 16, 32, CALL_TEAM)                          \
    GC_ROUTE_TEAM(T, whole, 64, 32, CALL_TEAM)
#define GC_ROUTE_BY_DTYPE(dt, experts, whole, CALL, CALL_TEAM, WARP)                                  \
    if (dt == GC_ROW_F32) { GC_ROUTE_BY_SIZE(float, experts, whole, CALL, CALL_TEAM, WARP) }          \
    if (dt == GC_ROW_BF16) { GC_ROUTE_BY_SIZE(__nv_bfloat16, experts, whole, CALL, CALL_TEAM, WARP) } \
    GC_ROUTE_BY_SIZE(__half, experts, whole, CALL, CALL_TEAM, WARP)

}  // namespace gcd
