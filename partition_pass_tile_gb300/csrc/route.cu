// route.cu -- every token's experts and their weights, the experts' counts and
// mean probabilities, the balance loss, and the gradient (gc_expert_route,
// gc_expert_route_grad).
//
// Per token, with x its logits (float32 of them, cleaned as gc_sample's):
// p = softmax(x); the choices are the top-k of x, equal values by index; their
// weights are p, or p over the choices' sum.  With n the tokens that have a
// choice, c[e] the pairs of expert e and f = c / sum c:
//     load = sum p / n,   loss = experts * sum f load,
//     dx   = p (a - <p, a>) + the weights' part,   a = dloss * experts / n * f.
// One read of the logits each way, and one write of the gradient.
//
// A token belongs to a group of 1 to 32 lanes; lane l of it holds the experts
// [l * V, (l + 1) * V) in registers, so that equal values go by lane and then
// by register, and the lane's sums over tokens of its experts' probabilities
// and counts stay in registers until the end.
#include "gc_rows.cuh"
#include "gc_rows_internal.h"

namespace {

using namespace gcd;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kResident = 3;       // CTAs per SM that a grid is sized for
constexpr int kJoinCluster = 8;    // CTAs that add up the CTAs' sums
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kNone = 0x007fffffu;  // order_bits(-inf): no expert
constexpr float kLog2e = 1.44269504f;
// Choices per thread that a CTA holds: a group of G lanes has at most 8 G
// experts, or is a warp with at most GC_MAX_TOPK choices.
constexpr int kPicks = 8;

struct Pick {
    float x;
    int32_t id;
};

// A group of lanes of a warp.
struct Group {
    uint32_t lanes, lane, mask;
    __device__ __forceinline__ explicit Group(uint32_t lanes_) : lanes(lanes_), lane(threadIdx.x & (lanes_ - 1))
    {
        mask = lanes == 32 ? kFull : ((1u << lanes) - 1u) << ((threadIdx.x & 31) - lane);
    }
    __device__ __forceinline__ uint32_t largest(uint32_t v) const
    {
        if (lanes == 32) return __reduce_max_sync(kFull, v);
        for (uint32_t o = lanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
    __device__ __forceinline__ float sum(float v) const
    {
        for (uint32_t o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
        return v;
    }
};

// This lane's logits of a token, -inf where there is none.
template <class T, int N, int V>
__device__ __forceinline__ void load_logits(const T *__restrict__ row, uint32_t first, uint32_t experts, bool live,
                                            float (&x)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += N) {
        if (live && first + i < experts) {
            const Piece<T, N> p = load_piece<T, N>(row + first + i);
#pragma unroll
            for (int e = 0; e < N; ++e) x[i + e] = sample_value(row_to_float(p.v[e]));
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x[i + e] = -INFINITY;
        }
    }
}

// What a CTA adds up of its tokens, per expert; sums[experts] and
// counts[experts + 1] (the tokens last) in shared or global memory.
struct Totals {
    float *sums;
    uint32_t *counts;
};

struct RouteOut {
    int32_t *counts;
    float *load, *loss;
};

// sum over threads of a CTA, of doubles; every thread calls it, thread 0 has it.
__device__ __forceinline__ double cta_sum(double v, double *s_warp)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kWarps; ++w) v += s_warp[w];
    return v;
}

// The group's sums -> the CTA's, in the order of the warps, eight registers at
// a time.  f(expert, sum, count) is called once per expert.
template <int V, class F>
__device__ __forceinline__ void join_warps(const Group &g, float (&sum)[V], uint32_t (&count)[V], uint32_t experts,
                                           float (*s_sum)[32 * 8], uint32_t (*s_count)[32 * 8], const F &f)
{
    const uint32_t warp = threadIdx.x >> 5;
    for (int base = 0; base < V; base += 8) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v < base || v >= base + 8) continue;
            float s = sum[v];
            uint32_t c = count[v];
            for (uint32_t o = g.lanes; o < 32; o <<= 1) {
                s += __shfl_xor_sync(kFull, s, o);
                c += __shfl_xor_sync(kFull, c, o);
            }
            if ((threadIdx.x & 31) < g.lanes) {
                s_sum[warp][g.lane * 8 + (v & 7)] = s;
                s_count[warp][g.lane * 8 + (v & 7)] = c;
            }
        }
        __syncthreads();
        const uint32_t e = (threadIdx.x >> 3) * V + base + (threadIdx.x & 7);  // lane threadIdx.x / 8
        if (threadIdx.x < g.lanes * 8 && e < experts) {
            float s = 0.0f;
            uint32_t c = 0;
            for (int w = 0; w < kWarps; ++w) {
                s += s_sum[w][threadIdx.x];
                c += s_count[w][threadIdx.x];
            }
            f(e, s, c);
        }
    }
    __syncthreads();
}

// `lanes`: of a group.  With out.counts NULL nothing is added up.  One CTA
// alone writes the results; several leave their sums in `part`.
template <class T, int N, int V>
__global__ void __launch_bounds__(kThreads)
route_kernel(const T *__restrict__ logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
             bool normalize, const uint8_t *__restrict__ mask, uint32_t lanes, int32_t *__restrict__ ids,
             float *__restrict__ weights, RouteOut out, Totals part)
{
    __shared__ Pick s_pick[kThreads * kPicks];
    __shared__ float s_sum[kWarps][32 * 8];
    __shared__ uint32_t s_count[kWarps][32 * 8];
    __shared__ double s_warp[kWarps];
    chain_start();
    const Group g(lanes);
    const uint32_t first = g.lane * V, groups = kThreads / lanes;
    Pick *pick = s_pick + (threadIdx.x - g.lane) * kPicks;
    float sum[V];
    uint32_t count[V], routed = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f, count[v] = 0;

    for (uint64_t base = uint64_t(blockIdx.x) * groups; base < tokens; base += uint64_t(gridDim.x) * groups) {
        const uint64_t t = base + threadIdx.x / lanes;
        const bool inside = t < tokens;
        const bool live = inside && (mask == nullptr || mask[t] != 0);
        float x[V];
        load_logits<T, N, V>(logits + t * stride, first, experts, live, x);
        uint32_t key[V], best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = order_bits(x[v]);
            best = max(best, key[v]);
        }
        uint32_t top = g.largest(best);
        const bool any = top > kNone;
        const float m = any ? order_value(top) : 0.0f;
        float total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = pow2((x[v] - m) * kLog2e);
            total += x[v];
        }
        total = g.sum(total);
        const float inverse = any ? 1.0f / total : 0.0f;
        routed += any && g.lane == 0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = fmaf(x[v], inverse, sum[v]);

        // the choices, one after another: the largest key of the group, of
        // equal ones the lowest lane's lowest
        for (uint32_t j = 0; j < topk; ++j) {
            if (j > 0) top = g.largest(best);
            const uint32_t have = __ballot_sync(kFull, best == top && top > kNone) & g.mask;
            if (have == 0) {
                if (g.lane == 0) pick[j] = Pick{-INFINITY, -1};
            } else if ((threadIdx.x & 31) == uint32_t(__ffs(have) - 1)) {
                best = 0;
                bool found = false;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!found && key[v] == top) {
                        found = true;
                        pick[j] = Pick{order_value(top), int32_t(first + v)};
                        key[v] = 0;
                    }
                    best = max(best, key[v]);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) count[v] += key[v] == 0;
        __syncwarp();
        float chosen = 0.0f;
        if (normalize) {
            for (uint32_t j = g.lane; j < topk; j += lanes) chosen += pow2((pick[j].x - m) * kLog2e);
            chosen = g.sum(chosen);
        }
        if (inside)
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const Pick c = pick[j];
                ids[t * topk + j] = c.id;
                weights[t * topk + j] =
                    c.id < 0 ? 0.0f : pow2((c.x - m) * kLog2e) / (normalize ? chosen : total);
            }
        __syncwarp();
    }
    if (out.counts == nullptr) return;

    if (gridDim.x > 1) {
        join_warps<V>(g, sum, count, experts, s_sum, s_count, [&](uint32_t e, float s, uint32_t c) {
            part.sums[size_t(blockIdx.x) * experts + e] = s;
            part.counts[size_t(blockIdx.x) * (experts + 1) + e] = c;
        });
        const double n = cta_sum(double(routed), s_warp);
        if (threadIdx.x == 0) part.counts[size_t(blockIdx.x) * (experts + 1) + experts] = uint32_t(n);
        return;
    }
    __shared__ double s_n;
    const double mine = cta_sum(double(routed), s_warp);
    if (threadIdx.x == 0) s_n = mine;
    __syncthreads();
    const double n = s_n;
    double pairs = 0.0, dot = 0.0;
    join_warps<V>(g, sum, count, experts, s_sum, s_count, [&](uint32_t e, float s, uint32_t c) {
        const double load = n > 0.0 ? double(s) / n : 0.0;
        out.counts[e] = int32_t(c);
        if (out.load) out.load[e] = float(load);
        pairs += double(c);
        dot += double(c) * load;
    });
    pairs = cta_sum(pairs, s_warp);
    dot = cta_sum(dot, s_warp);
    if (threadIdx.x == 0) {
        out.counts[experts] = int32_t(n);
        if (out.loss) *out.loss = pairs > 0.0 ? float(double(experts) * dot / pairs) : 0.0f;
    }
}

// The CTAs' sums, 32 experts at a time, each by eight threads that take every
// eighth CTA; one cluster, whose first CTA writes the loss.
__global__ void __cluster_dims__(kJoinCluster, 1, 1) __launch_bounds__(kThreads)
route_join_kernel(Totals part, uint32_t parts, uint32_t experts, RouteOut out)
{
    __shared__ double s_warp[kWarps];
    __shared__ double s_sum[kWarps][32];
    __shared__ uint32_t s_count[kWarps][32];
    __shared__ double s_got[2][kJoinCluster];
    const uint32_t rank = cluster_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    chain_wait();
    double n = 0.0;
    for (uint32_t c = threadIdx.x; c < parts; c += kThreads) n += double(part.counts[size_t(c) * (experts + 1) + experts]);
    n = cta_sum(n, s_warp);
    if (threadIdx.x == 0) s_warp[0] = n;
    __syncthreads();
    n = s_warp[0];
    double pairs = 0.0, dot = 0.0;
    for (uint32_t e0 = rank * 32; e0 < experts; e0 += kJoinCluster * 32) {
        const uint32_t e = e0 + lane;
        double s = 0.0;
        uint32_t k = 0;
        if (e < experts) {
#pragma unroll 8
            for (uint32_t c = warp; c < parts; c += kWarps) {
                s += double(part.sums[size_t(c) * experts + e]);
                k += part.counts[size_t(c) * (experts + 1) + e];
            }
        }
        __syncthreads();
        s_sum[warp][lane] = s;
        s_count[warp][lane] = k;
        __syncthreads();
        if (warp == 0 && e < experts) {
            for (int w = 1; w < kWarps; ++w) {
                s += s_sum[w][lane];
                k += s_count[w][lane];
            }
            const double load = n > 0.0 ? s / n : 0.0;
            out.counts[e] = int32_t(k);
            if (out.load) out.load[e] = float(load);
            pairs += double(k);
            dot += double(k) * load;
        }
    }
    pairs = cta_sum(pairs, s_warp);
    dot = cta_sum(dot, s_warp);
    cluster_sync();  // every CTA of the cluster runs
    if (threadIdx.x == 0) {
        peer_store(peer_address(&s_got[0][rank], 0), pairs);
        peer_store(peer_address(&s_got[1][rank], 0), dot);
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        pairs = dot = 0.0;
        for (int c = 0; c < kJoinCluster; ++c) {
            pairs += s_got[0][c];
            dot += s_got[1][c];
        }
        out.counts[experts] = int32_t(n);
        if (out.loss) *out.loss = pairs > 0.0 ? float(double(experts) * dot / pairs) : 0.0f;
    }
}

// The gradient: the softmax again, the row's two sums, and the row; then each
// choice's element once more with its own part, by the lane that has its id.
template <class T, int N, int V>
__global__ void __launch_bounds__(kThreads)
route_grad_kernel(const T *__restrict__ logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                  bool normalize, uint32_t lanes, const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                  const float *__restrict__ dweights, const float *__restrict__ dloss, T *__restrict__ dx,
                  size_t dx_stride)
{
    __shared__ Pick s_pick[kThreads * kPicks];
    __shared__ double s_warp[kWarps];
    __shared__ float s_factor;
    const Group g(lanes);
    const uint32_t first = g.lane * V, groups = kThreads / lanes;
    Pick *pick = s_pick + (threadIdx.x - g.lane) * kPicks;
    // a = factor * counts, by expert
    float a[V], factor = 0.0f;
    if (dloss != nullptr) {
        double pairs = 0.0;
        for (uint32_t e = threadIdx.x; e < experts; e += kThreads) pairs += double(max(counts[e], 0));
        pairs = cta_sum(pairs, s_warp);
        if (threadIdx.x == 0) {
            const double n = double(counts[experts]);
            s_factor = pairs > 0.0 && n > 0.0 ? float(double(*dloss) * double(experts) / (n * pairs)) : 0.0f;
        }
        __syncthreads();
        factor = s_factor;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = dloss != nullptr && first + v < experts ? factor * float(counts[first + v]) : 0.0f;

    for (uint64_t base = uint64_t(blockIdx.x) * groups; base < tokens; base += uint64_t(gridDim.x) * groups) {
        const uint64_t t = base + threadIdx.x / lanes;
        const bool inside = t < tokens;
        const bool live = inside && uint32_t(ids[t * topk]) < experts;
        const T *row = logits + t * stride;
        float p[V], m = -INFINITY;
        load_logits<T, N, V>(row, first, experts, live, p);
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, p[v]);
        const uint32_t top = g.largest(order_bits(m));
        m = top > kNone ? order_value(top) : 0.0f;
        float total = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = pow2((p[v] - m) * kLog2e);
            total += p[v];
            dot = fmaf(p[v], a[v], dot);
        }
        total = g.sum(total);
        const float inverse = total > 0.0f ? 1.0f / total : 0.0f;
        dot = g.sum(dot) * inverse;

        // the choices' weights and their gradients
        float chosen = 0.0f, inner = 0.0f;
        if (dweights != nullptr) {
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const uint32_t id = live ? uint32_t(ids[t * topk + j]) : ~0u;
                float w = 0.0f, d = 0.0f;
                if (id < experts) {
                    w = pow2((sample_value(row_to_float(row[id])) - m) * kLog2e) * inverse;
                    d = dweights[t * topk + j];
                }
                chosen += w;
                inner += w * d;
            }
            chosen = g.sum(chosen);
            inner = g.sum(inner);
            if (normalize) {
                inner = chosen > 0.0f ? inner / chosen : 0.0f;
            } else {
                dot += inner;
            }
            // pick: the id and what its choices add to its element
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const uint32_t id = live ? uint32_t(ids[t * topk + j]) : ~0u;
                Pick c{0.0f, -1};
                if (id < experts) {
                    const float w = pow2((sample_value(row_to_float(row[id])) - m) * kLog2e) * inverse;
                    const float d = dweights[t * topk + j];
                    c.id = int32_t(id);
                    c.x = normalize ? (chosen > 0.0f ? w / chosen * (d - inner) : 0.0f) : w * d;
                }
                pick[j] = c;
            }
        }
        if (inside) {
            T *to = dx + t * dx_stride;
#pragma unroll
            for (int i = 0; i < V; i += N) {
                if (first + i >= experts) break;
                Piece<T, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) o.v[e] = row_from_float<T>(p[i + e] * inverse * (a[i + e] - dot));
                store_piece<T, N>(to + first + i, o);
            }
        }
        __syncwarp();
        if (dweights != nullptr && live) {
            T *to = dx + t * dx_stride;
            for (uint32_t j = g.lane; j < topk; j += lanes) {
                const int32_t id = pick[j].id;
                if (id < 0) continue;
                // an id that occurs twice has both choices' parts, and both lanes write the same
                float part = 0.0f;
                for (uint32_t q = 0; q < topk; ++q)
                    if (pick[q].id == id) part += pick[q].x;
                const float w = pow2((sample_value(row_to_float(row[id])) - m) * kLog2e) * inverse;
                const float c = dloss != nullptr ? factor * float(counts[id]) : 0.0f;
                to[id] = row_from_float<T>(w * (c - dot) + part);
            }
        }
        __syncwarp();
    }
}

// Experts per lane and lanes per token: eight experts to a lane up to 256,
// more registers beyond.
struct Shape {
    int values;
    uint32_t lanes;
};

Shape shape_of(uint32_t experts)
{
    Shape s{8, 1};
    while (s.lanes < 32 && s.lanes * 8 < experts) s.lanes *= 2;
    while (s.lanes * uint32_t(s.values) < experts) s.values *= 2;
    return s;
}

uint32_t route_grid(uint32_t tokens, uint32_t lanes)
{
    const size_t need = gch::ceil_div(tokens, kThreads / lanes), most = gch::kSms * kResident;
    return uint32_t(need < most ? need : most);
}

template <class T, int N, int V>
cudaError_t run_route(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                      bool normalize, const uint8_t *mask, uint32_t lanes, int32_t *ids, float *weights,
                      const RouteOut &out, uint8_t *ws, cudaStream_t s)
{
    const uint32_t grid = tokens ? route_grid(tokens, lanes) : 1;
    const Totals part{reinterpret_cast<float *>(ws),
                      reinterpret_cast<uint32_t *>(ws + gch::align_up(size_t(grid) * experts * 4, 256))};
    route_kernel<T, N, V><<<grid, kThreads, 0, s>>>(static_cast<const T *>(logits), stride, tokens, experts, topk,
                                                    normalize, mask, lanes, ids, weights, out, part);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && out.counts && grid > 1)
        e = gch::launch_next(route_join_kernel, dim3(kJoinCluster), dim3(kThreads), 0, s, part, grid, experts, out);
    return e;
}

template <class T, int N, int V>
cudaError_t run_route_grad(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                           bool normalize, uint32_t lanes, const int32_t *ids, const int32_t *counts,
                           const float *dweights, const float *dloss, void *dx, size_t dx_stride, cudaStream_t s)
{
    route_grad_kernel<T, N, V><<<route_grid(tokens, lanes), kThreads, 0, s>>>(
        static_cast<const T *>(logits), stride, tokens, experts, topk, normalize, lanes, ids, counts, dweights, dloss,
        static_cast<T *>(dx), dx_stride);
    return cudaGetLastError();
}

// Pieces of 16 bytes where pointers, strides and experts allow it, else
// elements; V by the number of experts.
#define GC_ROUTE_BY_VALUES(T, N, values, CALL)          \
    switch (values) {                                   \
    case 8: return CALL(T, N, 8);                       \
    case 16: return CALL(T, N, 16);                     \
    case 32: return CALL(T, N, 32);                     \
    default: return CALL(T, N, 64);                     \
    }
#define GC_ROUTE_BY_PIECE(T, whole, values, CALL)                       \
    if (whole) { GC_ROUTE_BY_VALUES(T, int(16 / sizeof(T)), values, CALL) } \
    else { GC_ROUTE_BY_VALUES(T, 1, values, CALL) }
#define GC_ROUTE_BY_DTYPE(dt, whole, values, CALL)                              \
    if (dt == GC_ROW_F32) { GC_ROUTE_BY_PIECE(float, whole, values, CALL) }     \
    else if (dt == GC_ROW_BF16) { GC_ROUTE_BY_PIECE(__nv_bfloat16, whole, values, CALL) } \
    else { GC_ROUTE_BY_PIECE(__half, whole, values, CALL) }

}  // namespace

namespace gch {

size_t expert_route_workspace_bytes(size_t tokens, uint32_t experts)
{
    const uint32_t grid = tokens ? route_grid(uint32_t(tokens), shape_of(experts).lanes) : 1;
    if (grid == 1) return 256;
    return align_up(size_t(grid) * experts * 4, 256) + align_up(size_t(grid) * (experts + 1) * 4, 256);
}

cudaError_t launch_expert_route(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, gc_row_dtype dt,
                                uint32_t topk, bool normalize, const uint8_t *mask, int32_t *ids, float *weights,
                                int32_t *counts, float *load, float *loss, uint8_t *ws, cudaStream_t s)
{
    const Shape shape = shape_of(experts);
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const bool whole = ((uintptr_t(logits) | elem * (stride | experts)) & 15u) == 0;
    const RouteOut out{counts, load, loss};
#define GC_ROUTE_CALL(T, N, V) \
    run_route<T, N, V>(logits, stride, tokens, experts, topk, normalize, mask, shape.lanes, ids, weights, out, ws, s)
    GC_ROUTE_BY_DTYPE(dt, whole, shape.values, GC_ROUTE_CALL)
}

cudaError_t launch_expert_route_grad(const void *logits, size_t stride, uint32_t tokens, uint32_t experts,
                                     gc_row_dtype dt, uint32_t topk, bool normalize, const int32_t *ids,
                                     const int32_t *counts, const float *dweights, const float *dloss, void *dx,
                                     size_t dx_stride, cudaStream_t s)
{
    const Shape shape = shape_of(experts);
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const bool whole = ((uintptr_t(logits) | uintptr_t(dx) | elem * (stride | dx_stride | experts)) & 15u) == 0;
#define GC_ROUTE_GRAD_CALL(T, N, V)                                                                             \
    run_route_grad<T, N, V>(logits, stride, tokens, experts, topk, normalize, shape.lanes, ids, counts, dweights, \
                            dloss, dx, dx_stride, s)
    GC_ROUTE_BY_DTYPE(dt, whole, shape.values, GC_ROUTE_GRAD_CALL)
}

}  // namespace gch
