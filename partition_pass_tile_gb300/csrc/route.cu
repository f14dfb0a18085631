// route.cu -- every token's experts and their weights, the experts' counts and
// mean probabilities, and the balance loss (gc_expert_route).
//
// Per token, with x its logits (float32 of them, cleaned as gc_sample's):
// p = softmax(x); the choices are the top-k of x, equal values by index; their
// weights are p, or p over the choices' sum.  With n the tokens that have a
// choice, c[e] the pairs of expert e and f = c / sum c:
//     load = sum p / n,   loss = experts * sum f load.
//
// One read of the logits.  Lane l of a warp (of a group of lanes where experts
// are few) holds the experts [l * V, (l + 1) * V) of a token in registers, so
// that equal values go by lane and then by register; the lane's sums over
// tokens of its experts' probabilities stay in registers until the end, CTAs
// leave them in the workspace, and a cluster adds them up.
#include "gc_route.cuh"

namespace {

using namespace gcd;

constexpr int kJoinThreads = 1024;
constexpr int kJoinCluster = 8;    // CTAs that add up the CTAs' sums

// What CTAs have added up of their tokens, by CTA: sums[experts] and
// counts[experts + 1], the tokens last.
struct Totals {
    float *sums;
    uint32_t *counts;
};

struct RouteOut {
    int32_t *ids;
    float *weights;
    int32_t *counts;  // NULL: nothing is added up
    float *load, *loss;
};

// loss = experts * dot / pairs, dot the sum of counts * load.
__device__ __forceinline__ float loss_of(uint32_t experts, float dot, uint32_t pairs)
{
    return pairs > 0 ? float(experts) * dot / float(pairs) : 0.0f;
}

// A CTA's sums: to the workspace, or, if it is the only one, to the results.
// each(f) calls f(expert, sum, count) by some thread for every expert.  No
// double here: that pipe makes a chain of reductions of one CTA take 10 us.
template <int W, class Each>
__device__ __forceinline__ void finish(uint32_t experts, uint32_t routed, const RouteOut &out, const Totals &part,
                                       uint32_t *s_warp, const Each &each)
{
    const uint32_t n = cta_count<W>(routed, s_warp);
    if (gridDim.x > 1) {
        each([&](uint32_t e, float s, uint32_t c) {
            part.sums[size_t(blockIdx.x) * experts + e] = s;
            part.counts[size_t(blockIdx.x) * (experts + 1) + e] = c;
        });
        if (threadIdx.x == 0) part.counts[size_t(blockIdx.x) * (experts + 1) + experts] = n;
        return;
    }
    uint32_t pairs = 0;
    float dot = 0.0f;
    each([&](uint32_t e, float s, uint32_t c) {
        const float load = n > 0 ? s / float(n) : 0.0f;
        out.counts[e] = int32_t(c);
        if (out.load) out.load[e] = load;
        pairs += c;
        dot = fmaf(float(c), load, dot);
    });
    pairs = cta_count<W>(pairs, s_warp);
    dot = cta_sum<W>(dot, s_warp);
    if (threadIdx.x == 0) {
        out.counts[experts] = int32_t(n);
        if (out.loss) *out.loss = loss_of(experts, dot, pairs);
    }
}

// ---------------------------------------------------------------- a warp to a token

template <int V>
constexpr int kWarpThreads = V <= 8 ? 512 : 256;
template <int V>
constexpr int kWarpResident = V <= 16 ? 2 : 1;  // CTAs per SM
constexpr uint32_t kCandidates = 64;

// A bit for each of a lane's experts.
template <int V>
struct Bits {
    using Type = typename std::conditional<(V > 32), uint64_t, uint32_t>::type;
    static __device__ __forceinline__ uint32_t count(Type b) { return V > 32 ? __popcll(b) : __popc(uint32_t(b)); }
    static __device__ __forceinline__ int lowest(Type b) { return (V > 32 ? __ffsll(b) : __ffs(uint32_t(b))) - 1; }
};

// The choices.  A lower bound of the k-th largest logit is the k-th largest of
// the lanes' largest: k warp-wide maxima.  The logits not below it, hardly more
// than k, are listed, one to a lane, and ranked by comparing each with all.
// Where they are more than a warp (many closed experts, equal values, large k)
// the choices are taken one after another.  131072 tokens of 256 float32, top-8:
// TIME us, against 162 one after another.
template <class T, int N, int V>
__global__ void __launch_bounds__(kWarpThreads<V>, kWarpResident<V>)
route_warp_kernel(const T *__restrict__ logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                  bool normalize, const uint8_t *__restrict__ mask, RouteOut out, Totals part)
{
    constexpr int kWarps = kWarpThreads<V> / 32;
    constexpr int kSlots = V < 8 ? V : 8;
    __shared__ uint32_t s_id[kWarps][kCandidates];
    __shared__ uint4 s_key[kWarps][kCandidates / 4];
    __shared__ float s_sum[kWarps][32 * kSlots];
    __shared__ uint32_t s_count[GC_MAX_EXPERTS];
    __shared__ uint32_t s_warp[kWarps];
    chain_start();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = lane * V;
    for (uint32_t e = threadIdx.x; e < experts; e += kWarpThreads<V>) s_count[e] = 0;
    __syncthreads();
    uint32_t *id = s_id[warp], *key = reinterpret_cast<uint32_t *>(s_key[warp]);
    float sum[V];
    uint32_t routed = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;

    const uint64_t step = uint64_t(gridDim.x) * kWarps;
    Logits<T, N, V> next;
    auto fetch = [&](uint64_t t) {
        next.load(logits + t * stride, first, experts, t < tokens && (mask == nullptr || mask[t] != 0));
    };
    uint64_t t = uint64_t(blockIdx.x) * kWarps + warp;
    fetch(t);
    for (; t < tokens; t += step) {
        float x[V], w[V];
        next.values(x);
        fetch(t + step);
        Exponent exponent;
        uint32_t top, left;
        const float total = warp_weights(x, w, exponent, top, left);
        int32_t *ids = out.ids + t * topk;
        float *weights = out.weights + t * topk;
        if (!(total > 0.0f)) {
            for (uint32_t j = lane; j < topk; j += 32) ids[j] = -1, weights[j] = 0.0f;
            continue;
        }
        ++routed;
        const float inverse = inverse_of(total);
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = fmaf(w[v], inverse, sum[v]);

        // a bound that at least k logits reach
        const uint32_t most = left;
        uint32_t bound = top;
        for (uint32_t j = 1; j < topk && bound > kRouteNone; ++j) {
            left = left == bound ? 0u : left;
            bound = __reduce_max_sync(kRouteFull, left);
        }
        const float least = order_value(max(bound, kRouteNone + 1));
        using Mask = typename Bits<V>::Type;
        Mask which = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) which |= x[v] >= least ? Mask(1) << v : Mask(0);
        const uint32_t mine = Bits<V>::count(which);
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kRouteFull, upto, o);
            if (lane >= uint32_t(o)) upto += y;
        }
        uint32_t n = __shfl_sync(kRouteFull, upto, 31), rank = lane;
        if (n <= 32) {
            // listed by id; read again, which spares finding them among the registers
            for (uint32_t at = upto - mine; which; which &= which - 1, ++at) id[at] = first + Bits<V>::lowest(which);
            key[lane] = 0;
            __syncwarp();
            uint32_t own = 0;
            if (lane < n) {
                own = order_bits(sample_value(row_to_float(logits[t * stride + id[lane]])));
                key[lane] = own;
            }
            __syncwarp();
            // before it: the larger ones, and the equal ones listed before it
            rank = 0;
            for (uint32_t c = 0; c < n; c += 4) {
                const uint4 k = s_key[warp][c / 4];
                rank += k.x >= own + (c >= lane);
                rank += k.y >= own + (c + 1 >= lane);
                rank += k.z >= own + (c + 2 >= lane);
                rank += k.w >= own + (c + 3 >= lane);
            }
            if (lane >= n) rank = ~0u;
        } else {
            // one after another: a lane's largest, and which of its logits are left
            Mask rest = ~Mask(0);
            left = most;
            for (n = 0; n < topk; ++n) {
                if (n > 0) top = __reduce_max_sync(kRouteFull, left);
                if (top <= kRouteNone) break;
                if (lane == uint32_t(__ffs(__ballot_sync(kRouteFull, left == top)) - 1)) {
                    left = 0;
                    bool found = false;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (!(rest >> v & 1u)) continue;
                        const uint32_t k = order_bits(x[v]);
                        if (!found && k == top) {
                            found = true;
                            rest &= ~(Mask(1) << v);
                            id[n] = first + v;
                            key[n] = top;
                        } else {
                            left = max(left, k);
                        }
                    }
                }
            }
            __syncwarp();
        }
        // n listed, ranked or in order
        const uint32_t listed = n;
        const bool own_one = lane < listed && rank < topk, other = lane + 32 < listed;
        const float first_w = own_one ? exponent.weight(order_value(key[lane])) : 0.0f;
        const float other_w = other ? exponent.weight(order_value(key[lane + 32])) : 0.0f;
        const float scale = normalize ? inverse_of(warp_sum(first_w + other_w)) : inverse;
        if (own_one) {
            ids[rank] = int32_t(id[lane]);
            weights[rank] = first_w * scale;
            if (out.counts) atomicAdd(&s_count[id[lane]], 1u);
        }
        if (other) {
            ids[lane + 32] = int32_t(id[lane + 32]);
            weights[lane + 32] = other_w * scale;
            if (out.counts) atomicAdd(&s_count[id[lane + 32]], 1u);
        }
        for (uint32_t j = listed + lane; j < topk; j += 32) ids[j] = -1, weights[j] = 0.0f;
        __syncwarp();
    }
    if (out.counts == nullptr) return;

    finish<kWarps>(experts, lane == 0 ? routed : 0u, out, part, s_warp, [&](const auto &f) {
        for (int base = 0; base < V; base += kSlots) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v >= base && v < base + kSlots) s_sum[warp][lane * kSlots + (v & (kSlots - 1))] = sum[v];
            __syncthreads();
            const uint32_t e = threadIdx.x / kSlots * V + base + threadIdx.x % kSlots;
            if (threadIdx.x < 32 * kSlots && e < experts) {
                float s = 0.0f;
                for (int w = 0; w < kWarps; ++w) s += s_sum[w][threadIdx.x];
                f(e, s, s_count[e]);
            }
        }
        __syncthreads();
    });
}

// ---------------------------------------------------------------- a group to a token

constexpr int kGroupThreads = 256;
constexpr int kGroupResident = 3;  // CTAs per SM

// The choices one after another: the largest key of the group, of equal ones the
// lowest lane's lowest.
template <class T, int N>
__global__ void __launch_bounds__(kGroupThreads)
route_group_kernel(const T *__restrict__ logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                   bool normalize, const uint8_t *__restrict__ mask, uint32_t lanes, RouteOut out, Totals part)
{
    constexpr int V = kGroupValues, kWarps = kGroupThreads / 32;
    // topk <= experts <= 8 lanes
    __shared__ Pick s_pick[kGroupThreads * V];
    __shared__ float s_sum[kWarps][4 * V];
    __shared__ uint32_t s_count[kWarps][4 * V];
    __shared__ uint32_t s_warp[kWarps];
    chain_start();
    const Group g(lanes);
    const uint32_t first = g.lane * V, groups = kGroupThreads / lanes;
    Pick *pick = s_pick + (threadIdx.x - g.lane) * V;
    float sum[V];
    uint32_t count[V], routed = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f, count[v] = 0;

    for (uint64_t base = uint64_t(blockIdx.x) * groups; base < tokens; base += uint64_t(gridDim.x) * groups) {
        const uint64_t t = base + threadIdx.x / lanes;
        const bool inside = t < tokens;
        Logits<T, N, V> row;
        row.load(logits + t * stride, first, experts, inside && (mask == nullptr || mask[t] != 0));
        float x[V];
        uint32_t key[V], best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = sample_value(row[v]);
            key[v] = order_bits(x[v]);
            best = max(best, key[v]);
        }
        uint32_t top = g.largest(best);
        const bool any = top > kRouteNone;
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

        for (uint32_t j = 0; j < topk; ++j) {
            if (j > 0) top = g.largest(best);
            const uint32_t have = __ballot_sync(kRouteFull, best == top && top > kRouteNone) & g.mask;
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
                out.ids[t * topk + j] = c.id;
                out.weights[t * topk + j] =
                    c.id < 0 ? 0.0f : pow2((c.x - m) * kLog2e) / (normalize ? chosen : total);
            }
        __syncwarp();
    }
    if (out.counts == nullptr) return;

    finish<kWarps>(experts, routed, out, part, s_warp, [&](const auto &f) {
        const uint32_t warp = threadIdx.x >> 5;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = sum[v];
            uint32_t c = count[v];
            for (uint32_t o = g.lanes; o < 32; o <<= 1) {
                s += __shfl_xor_sync(kRouteFull, s, o);
                c += __shfl_xor_sync(kRouteFull, c, o);
            }
            if ((threadIdx.x & 31) < g.lanes) {
                s_sum[warp][first + v] = s;
                s_count[warp][first + v] = c;
            }
        }
        __syncthreads();
        if (threadIdx.x < experts) {
            float s = 0.0f;
            uint32_t c = 0;
            for (int w = 0; w < kWarps; ++w) {
                s += s_sum[w][threadIdx.x];
                c += s_count[w][threadIdx.x];
            }
            f(threadIdx.x, s, c);
        }
        __syncthreads();
    });
}

// ---------------------------------------------------------------- the CTAs' sums

// 32 experts to a CTA at a time, a warp to every 32nd of the CTAs; one cluster,
// whose first CTA writes the loss.
__global__ void __cluster_dims__(kJoinCluster, 1, 1) __launch_bounds__(kJoinThreads)
route_join_kernel(Totals part, uint32_t parts, uint32_t experts, RouteOut out)
{
    constexpr int kWarps = kJoinThreads / 32;
    __shared__ uint32_t s_warp[kWarps];
    __shared__ float s_sum[kWarps][32];
    __shared__ uint32_t s_count[kWarps][32];
    __shared__ float s_dot[kJoinCluster];
    __shared__ uint32_t s_pairs[kJoinCluster];
    const uint32_t rank = cluster_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    chain_wait();
    uint32_t n = 0;
    for (uint32_t c = threadIdx.x; c < parts; c += kJoinThreads) n += part.counts[size_t(c) * (experts + 1) + experts];
    n = cta_count<kWarps>(n, s_warp);
    uint32_t pairs = 0;
    float dot = 0.0f;
    for (uint32_t e0 = rank * 32; e0 < experts; e0 += kJoinCluster * 32) {
        const uint32_t e = e0 + lane;
        float s = 0.0f;
        uint32_t k = 0;
        if (e < experts) {
#pragma unroll 10
            for (uint32_t c = warp; c < parts; c += kWarps) {
                s += part.sums[size_t(c) * experts + e];
                k += part.counts[size_t(c) * (experts + 1) + e];
            }
        }
        __syncthreads();
        s_sum[warp][lane] = s;
        s_count[warp][lane] = k;
        __syncthreads();
        // a warp to an expert
        const uint32_t mine = e0 + warp;
        if (mine < experts) {
            s = warp_sum(s_sum[lane][warp]);
            k = __reduce_add_sync(kRouteFull, s_count[lane][warp]);
            if (lane == 0) {
                const float load = n > 0 ? s / float(n) : 0.0f;
                out.counts[mine] = int32_t(k);
                if (out.load) out.load[mine] = load;
                pairs += k;
                dot = fmaf(float(k), load, dot);
            }
        }
    }
    pairs = cta_count<kWarps>(pairs, s_warp);
    dot = cta_sum<kWarps>(dot, s_warp);
    cluster_sync();  // every CTA of the cluster runs
    if (threadIdx.x == 0) {
        peer_store(peer_address(&s_dot[rank], 0), __float_as_uint(dot));
        peer_store(peer_address(&s_pairs[rank], 0), pairs);
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        pairs = 0, dot = 0.0f;
        for (int c = 0; c < kJoinCluster; ++c) {
            pairs += s_pairs[c];
            dot += s_dot[c];
        }
        out.counts[experts] = int32_t(n);
        if (out.loss) *out.loss = loss_of(experts, dot, pairs);
    }
}

// CTAs: as many as run at a time, each with the tokens of its warps or groups at
// least once; one alone, which spares the second launch, where it has them at
// most kAlone times (24 tokens of 64 experts: ALONE1 us against ALONE2 by two launches;
// 128 tokens ALONE3 against ALONE4).
constexpr size_t kAlone = 4;

uint32_t route_grid(uint32_t tokens, uint32_t experts)
{
    const bool warps = experts > kSmallExperts;
    const int v = route_values(experts);
    const size_t each = warps ? (v <= 8 ? kWarpThreads<8> : kWarpThreads<64>) / 32 : kGroupThreads / route_lanes(experts);
    const size_t resident = warps ? (v <= 16 ? kWarpResident<8> : kWarpResident<64>) : kGroupResident;
    const size_t need = gch::ceil_div(tokens, each), most = gch::kSms * resident;
    return uint32_t(need <= kAlone ? 1 : need < most ? need : most);
}

Totals totals_in(uint8_t *ws, uint32_t grid, uint32_t experts)
{
    return Totals{reinterpret_cast<float *>(ws),
                  reinterpret_cast<uint32_t *>(ws + gch::align_up(size_t(grid) * experts * 4, 256))};
}

cudaError_t join(const Totals &part, uint32_t grid, uint32_t experts, const RouteOut &out, cudaStream_t s)
{
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && out.counts && grid > 1)
        e = gch::launch_next(route_join_kernel, dim3(kJoinCluster), dim3(kJoinThreads), 0, s, part, grid, experts, out);
    return e;
}

template <class T, int N>
cudaError_t run_group(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                      bool normalize, const uint8_t *mask, const RouteOut &out, uint8_t *ws, cudaStream_t s)
{
    const uint32_t grid = route_grid(tokens, experts);
    const Totals part = totals_in(ws, grid, experts);
    route_group_kernel<T, N><<<grid, kGroupThreads, 0, s>>>(static_cast<const T *>(logits), stride, tokens, experts,
                                                            topk, normalize, mask, route_lanes(experts), out, part);
    return join(part, grid, experts, out, s);
}

template <class T, int N, int V>
cudaError_t run_warp(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                     bool normalize, const uint8_t *mask, const RouteOut &out, uint8_t *ws, cudaStream_t s)
{
    const uint32_t grid = route_grid(tokens, experts);
    const Totals part = totals_in(ws, grid, experts);
    route_warp_kernel<T, N, V><<<grid, kWarpThreads<V>, 0, s>>>(static_cast<const T *>(logits), stride, tokens,
                                                                experts, topk, normalize, mask, out, part);
    return join(part, grid, experts, out, s);
}

}  // namespace

namespace gch {

size_t expert_route_workspace_bytes(size_t tokens, uint32_t experts)
{
    const uint32_t grid = route_grid(uint32_t(tokens), experts);
    if (grid == 1) return 256;
    return align_up(size_t(grid) * experts * 4, 256) + align_up(size_t(grid) * (experts + 1) * 4, 256);
}

cudaError_t launch_expert_route(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, gc_row_dtype dt,
                                uint32_t topk, bool normalize, const uint8_t *mask, int32_t *ids, float *weights,
                                int32_t *counts, float *load, float *loss, uint8_t *ws, cudaStream_t s)
{
    const size_t elem = dt == GC_ROW_F32 ? 4 : 2;
    const bool whole = ((uintptr_t(logits) | elem * (stride | experts)) & 15u) == 0;
    const RouteOut out{ids, weights, counts, load, loss};
#define GC_ROUTE_CALL(T, N) run_group<T, N>(logits, stride, tokens, experts, topk, normalize, mask, out, ws, s)
#define GC_ROUTE_CALL_WARP(T, N, V) run_warp<T, N, V>(logits, stride, tokens, experts, topk, normalize, mask, out, ws, s)
    GC_ROUTE_BY_DTYPE(dt, experts, whole, GC_ROUTE_CALL, GC_ROUTE_CALL_WARP)
}

}  // namespace gch
