// route_grad.cu -- the gradient of routing with respect to the logits
// (gc_expert_route_grad).
//
// With p = softmax(x) of a token, f the experts' shares of the choices, w the
// weights of its choices and g their gradients:
//     dx = p (a - <p, a>) + the weights' part,   a = dloss * experts / n * f.
// The softmax is taken again: one read of the logits, one write of the
// gradient.  The row is written without the weights' part of its choices, and
// then each choice's element once more, whole, by the lane that has the choice.
#include "gc_route.cuh"

namespace {

using namespace gcd;

struct Grad {
    uint32_t tokens, experts, topk;
    size_t stride, dx_stride;
    bool normalize;
    const int32_t *ids, *counts;
    const float *dweights, *dloss;  // either may be NULL
};

// dloss * experts / (n * pairs): a = factor * counts.  Every thread has it.
template <int W>
__device__ __forceinline__ float loss_factor(const Grad &a, uint32_t *s_warp)
{
    if (a.dloss == nullptr) return 0.0f;
    uint32_t pairs = 0;
    for (uint32_t e = threadIdx.x; e < a.experts; e += W * 32) pairs += uint32_t(max(a.counts[e], 0));
    pairs = cta_count<W>(pairs, s_warp);
    const int32_t n = a.counts[a.experts];
    return pairs > 0 && n > 0 ? *a.dloss * float(a.experts) / float(n) / float(pairs) : 0.0f;
}

// ---------------------------------------------------------------- a team to a token

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int V>
constexpr int kResident = V <= 4 ? 4 : V == 8 ? 3 : V == 16 ? 2 : 1;  // CTAs per SM

// The next token's logits and choices are on their way while one is computed.
// 131072 tokens of 64 float32, 128 bf16 and 256 float32 by teams of 16: 24, 29
// and 54 us (the last 75% of the copy rate); by whole warps, which pay for every
// token what does not depend on its experts, 59, 70 and 64.
template <class T, int N, int V, int G>
__global__ void __launch_bounds__(kThreads, kResident<V>)
route_grad_team_kernel(const T *__restrict__ logits, T *__restrict__ dx, Grad a)
{
    constexpr int kTeams = 32 / G;
    __shared__ Pick s_pick[kWarps * kTeams][GC_MAX_TOPK];
    __shared__ uint32_t s_warp[kWarps];
    const uint32_t lane = threadIdx.x & (G - 1), team = threadIdx.x / G, first = lane * N;
    using Row = Logits<T, N, V, G>;
    Pick *pick = s_pick[team];
    const float factor = loss_factor<kWarps>(a, s_warp);
    float share[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t e = Row::expert(first, v);
        share[v] = a.dloss && e < a.experts ? factor * float(a.counts[e]) : 0.0f;
    }
    const bool few = a.topk <= G;  // a choice to a lane

    const uint64_t step = uint64_t(gridDim.x) * kWarps * kTeams;
    uint64_t base = uint64_t(blockIdx.x) * kWarps * kTeams;
    Row next;
    uint32_t next_id = ~0u;
    float next_g = 0.0f;
    auto fetch = [&](uint64_t at) {
        next.load(logits + at * a.stride, first, a.experts, at < a.tokens);
        next_id = ~0u;
        if (at < a.tokens && lane < a.topk) {
            next_id = uint32_t(a.ids[at * a.topk + lane]);
            if (a.dweights) next_g = a.dweights[at * a.topk + lane];
        }
    };
    fetch(base + team);
    for (; base < a.tokens; base += step) {
        const uint64_t t = base + team;
        const bool inside = t < a.tokens;
        float x[V];
        next.values(x);
        const uint32_t id = next_id < a.experts ? next_id : ~0u;
        const float g = id != ~0u ? next_g : 0.0f;
        fetch(t + step);
        T *to = dx + t * a.dx_stride;
        const T *row = logits + t * a.stride;
        // a token without a choice has a row of zeros
        const bool live = __shfl_sync(kRouteFull, id, 0, G) != ~0u;
        float w[V];
        Exponent exponent;
        uint32_t top, best;
        const float total = team_weights<G>(x, w, exponent, top, best);
        const float inverse = live && total > 0.0f ? inverse_of(total) : 0.0f;
        float dot = 0.0f;
        if (a.dloss) {
#pragma unroll
            for (int v = 0; v < V; ++v) dot = fmaf(w[v], share[v], dot);
            dot = team_sum<G>(dot) * inverse;
        }
        // the choices' weights, and what they add to their elements
        float mine = 0.0f, part = 0.0f;
        if (a.dweights && few) {
            if (live && id != ~0u) mine = exponent.weight(row_to_float(row[id])) * inverse;
            float inner = team_sum<G>(mine * g);
            if (a.normalize) {
                const float chosen = team_sum<G>(mine), scale = chosen > 0.0f ? inverse_of(chosen) : 0.0f;
                part = mine * scale * (g - inner * scale);
            } else {
                dot += inner;
                part = mine * g;
            }
        } else if (a.dweights) {
            float chosen = 0.0f, inner = 0.0f;
            for (uint32_t j = lane; j < a.topk; j += G) {
                const uint32_t e = live ? uint32_t(a.ids[t * a.topk + j]) : ~0u;
                Pick c{0.0f, -1};
                if (e < a.experts) c = Pick{exponent.weight(row_to_float(row[e])) * inverse, int32_t(e)};
                pick[j] = c;
                chosen += c.x;
                if (c.id >= 0) inner += c.x * a.dweights[t * a.topk + j];
            }
            chosen = team_sum<G>(chosen);
            inner = team_sum<G>(inner);
            const float scale = chosen > 0.0f ? inverse_of(chosen) : 0.0f;
            if (a.normalize) inner *= scale;
            else dot += inner;
            for (uint32_t j = lane; j < a.topk; j += G)
                if (pick[j].id >= 0)
                    pick[j].x *= a.normalize ? scale * (a.dweights[t * a.topk + j] - inner) : a.dweights[t * a.topk + j];
        }
        if (inside) {
#pragma unroll
            for (int i = 0; i < V; i += N) {
                const uint32_t at = Row::expert(first, i);
                if (at >= a.experts) break;
                Piece<T, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    o.v[e] = row_from_float<T>(live ? w[i + e] * inverse * (share[i + e] - dot) : 0.0f);
                store_piece<T, N>(to + at, o);
            }
        }
        if (!a.dweights) continue;
        __syncwarp();
        // An id that occurs twice has both choices' parts, and both lanes write the same.
        if (few) {
            const bool has = live && id != ~0u;
            const uint32_t same = __match_any_sync(kRouteFull, has ? (threadIdx.x & 31 & ~(G - 1)) << 16 | id : 0x80000000u | lane);
            if (__any_sync(kRouteFull, has && (same & (same - 1)) != 0)) {
                const float own = part;
                part = 0.0f;
                for (int q = 0; q < 32; ++q) {
                    const float other = __shfl_sync(kRouteFull, own, q);
                    if (same >> q & 1u) part += other;
                }
            }
            if (has) {
                const float c = a.dloss ? factor * float(a.counts[id]) : 0.0f;
                to[id] = row_from_float<T>(mine * (c - dot) + part);
            }
        } else {
            for (uint32_t j = lane; j < a.topk; j += G) {
                const int32_t e = live ? pick[j].id : -1;
                if (e < 0) continue;
                float both = 0.0f;
                for (uint32_t q = 0; q < a.topk; ++q)
                    if (pick[q].id == e) both += pick[q].x;
                const float c = a.dloss ? factor * float(a.counts[e]) : 0.0f;
                to[e] = row_from_float<T>(exponent.weight(row_to_float(row[e])) * inverse * (c - dot) + both);
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- a group to a token

constexpr int kGroupResident = 4;  // CTAs per SM

template <class T, int N>
__global__ void __launch_bounds__(kThreads)
route_grad_group_kernel(const T *__restrict__ logits, T *__restrict__ dx, Grad a, uint32_t lanes)
{
    constexpr int V = kGroupValues;
    __shared__ Pick s_pick[kThreads * V];
    __shared__ uint32_t s_warp[kWarps];
    const Group g(lanes);
    const uint32_t first = g.lane * V, groups = kThreads / lanes, experts = a.experts, topk = a.topk;
    Pick *pick = s_pick + (threadIdx.x - g.lane) * V;
    const float factor = loss_factor<kWarps>(a, s_warp);
    float share[V];
#pragma unroll
    for (int v = 0; v < V; ++v) share[v] = a.dloss && first + v < experts ? factor * float(a.counts[first + v]) : 0.0f;

    for (uint64_t base = uint64_t(blockIdx.x) * groups; base < a.tokens; base += uint64_t(gridDim.x) * groups) {
        const uint64_t t = base + threadIdx.x / lanes;
        const bool inside = t < a.tokens;
        const bool live = inside && uint32_t(a.ids[t * topk]) < experts;
        const T *row = logits + t * a.stride;
        Logits<T, N, V, 1> x;
        x.load(row, first, experts, live);
        float p[V], m = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = sample_value(x[v]);
            m = fmaxf(m, p[v]);
        }
        const uint32_t top = g.largest(order_bits(m));
        m = top > kRouteNone ? order_value(top) : 0.0f;
        float total = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = pow2((p[v] - m) * kLog2e);
            total += p[v];
            dot = fmaf(p[v], share[v], dot);
        }
        total = g.sum(total);
        const float inverse = total > 0.0f ? 1.0f / total : 0.0f;
        dot = g.sum(dot) * inverse;

        // the choices' weights and their gradients
        float chosen = 0.0f, inner = 0.0f;
        if (a.dweights != nullptr) {
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const uint32_t id = live ? uint32_t(a.ids[t * topk + j]) : ~0u;
                Pick c{0.0f, -1};
                if (id < experts) {
                    c = Pick{pow2((sample_value(row_to_float(row[id])) - m) * kLog2e) * inverse, int32_t(id)};
                    inner += c.x * a.dweights[t * topk + j];
                }
                pick[j] = c;
                chosen += c.x;
            }
            chosen = g.sum(chosen);
            inner = g.sum(inner);
            const float scale = chosen > 0.0f ? 1.0f / chosen : 0.0f;
            if (a.normalize) inner *= scale;
            else dot += inner;
            // pick: the id and what its choice adds to its element
            for (uint32_t j = g.lane; j < topk; j += lanes)
                if (pick[j].id >= 0)
                    pick[j].x *= a.normalize ? scale * (a.dweights[t * topk + j] - inner) : a.dweights[t * topk + j];
        }
        T *to = dx + t * a.dx_stride;
        if (inside) {
#pragma unroll
            for (int i = 0; i < V; i += N) {
                if (first + i >= experts) break;
                Piece<T, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) o.v[e] = row_from_float<T>(p[i + e] * inverse * (share[i + e] - dot));
                store_piece<T, N>(to + first + i, o);
            }
        }
        __syncwarp();
        if (a.dweights != nullptr && live) {
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const int32_t id = pick[j].id;
                if (id < 0) continue;
                float part = 0.0f;
                for (uint32_t q = 0; q < topk; ++q)
                    if (pick[q].id == id) part += pick[q].x;
                const float w = pow2((sample_value(row_to_float(row[id])) - m) * kLog2e) * inverse;
                const float c = a.dloss != nullptr ? factor * float(a.counts[id]) : 0.0f;
                to[id] = row_from_float<T>(w * (c - dot) + part);
            }
        }
        __syncwarp();
    }
}

uint32_t grid_of(uint32_t tokens, size_t each, size_t resident)
{
    const size_t need = gch::ceil_div(tokens, each), most = gch::kSms * resident;
    return uint32_t(need < most ? need : most);
}

template <class T, int N>
cudaError_t run_group(const void *logits, void *dx, const Grad &a, cudaStream_t s)
{
    const uint32_t lanes = route_lanes(a.experts);
    route_grad_group_kernel<T, N><<<grid_of(a.tokens, kThreads / lanes, kGroupResident), kThreads, 0, s>>>(
        static_cast<const T *>(logits), static_cast<T *>(dx), a, lanes);
    return cudaGetLastError();
}

template <class T, int N, int V, int G>
cudaError_t run_team(const void *logits, void *dx, const Grad &a, cudaStream_t s)
{
    route_grad_team_kernel<T, N, V, G><<<grid_of(a.tokens, kThreads / G, kResident<V>), kThreads, 0, s>>>(
        static_cast<const T *>(logits), static_cast<T *>(dx), a);
    return cudaGetLastError();
}

}  // namespace

namespace gch {

cudaError_t launch_expert_route_grad(const void *logits, size_t stride, uint32_t tokens, uint32_t experts,
                                     gc_row_dtype dt, uint32_t topk, bool normalize, const int32_t *ids,
                                     const int32_t *counts, const float *dweights, const float *dloss, void *dx,
                                     size_t dx_stride, cudaStream_t s)
{
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const bool whole = ((uintptr_t(logits) | uintptr_t(dx) | elem * (stride | dx_stride | experts)) & 15u) == 0;
    const Grad a{tokens, experts, topk, stride, dx_stride, normalize, ids, counts, dweights, dloss};
#define GC_ROUTE_GRAD_CALL(T, N) run_group<T, N>(logits, dx, a, s)
#define GC_ROUTE_GRAD_CALL_TEAM(T, N, V, G) run_team<T, N, V, G>(logits, dx, a, s)
    GC_ROUTE_BY_DTYPE(dt, experts, whole, GC_ROUTE_GRAD_CALL, GC_ROUTE_GRAD_CALL_TEAM, GC_ROUTE_NO_WARP)
}

}  // namespace gch
