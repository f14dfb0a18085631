// route.cu -- every token's experts and their weights, the experts' counts and
// mean probabilities, and the balance loss (gc_expert_route).
//
// Per token, with x its logits (float32 of them, cleaned as gc_sample's):
// p = softmax(x); the choices are the top-k of x, equal values by index; their
// weights are p, or p over the choices' sum.  With n the tokens that have a
// choice, c[e] the pairs of expert e and f = c / sum c:
//     load = sum p / n,   loss = experts * sum f load.
//
// One read of the logits.  A token's experts lie in the registers of a team of 16
// or 32 lanes, or of a smaller group where experts are few; the lanes' sums over
// tokens of their experts' probabilities stay there until the end, CTAs leave
// them in the workspace, and a cluster adds them up.
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

// ---------------------------------------------------------------- a team to a token

template <int V>
constexpr int kTeamThreads = V <= 8 ? 512 : 256;
template <int V>
constexpr int kTeamResident = V <= 8 ? 2 : V == 16 ? 3 : 1;  // CTAs per SM
constexpr uint32_t kCandidates = 64;
// Choices that a team of 16 lanes makes: the bound below is one of its lanes'
// largest, and the candidates have to be hardly more than the lanes.
constexpr uint32_t kHalfTopk = 12;

// A bit for each of a lane's experts.
template <int V>
struct Bits {
    using Type = typename std::conditional<(V > 32), uint64_t, uint32_t>::type;
    static __device__ __forceinline__ uint32_t count(Type b) { return V > 32 ? __popcll(b) : __popc(uint32_t(b)); }
    static __device__ __forceinline__ int lowest(Type b) { return (V > 32 ? __ffsll(b) : __ffs(uint32_t(b))) - 1; }
};

// The k-th largest of a team's values, k <= G: of 16 lanes by sorting them (ten
// exchanges), of 32 by taking the largest off k - 1 times.
template <int G>
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, uint32_t top, uint32_t k)
{
    if constexpr (G == 32) {
        uint32_t bound = top;
        for (uint32_t j = 1; j < k && bound > kRouteNone; ++j) {
            v = v == bound ? 0u : v;
            bound = __reduce_max_sync(kRouteFull, v);
        }
        return bound;
    } else {
        const uint32_t lane = threadIdx.x & (G - 1);
#pragma unroll
        for (uint32_t size = 2; size <= G; size <<= 1)
#pragma unroll
            for (uint32_t o = size / 2; o > 0; o >>= 1) {
                const uint32_t other = __shfl_xor_sync(kRouteFull, v, o);
                // in descending order at the end
                v = ((lane & o) != 0) == ((lane & size) != 0) ? max(v, other) : min(v, other);
            }
        return __shfl_sync(kRouteFull, v, k - 1, G);
    }
}

// The choices.  A lower bound of the k-th largest logit is the k-th largest of
// the lanes' largest.  The logits not below it, hardly more than k, are listed,
// one to a lane, and ranked by comparing each with all.  Where they are more
// than the lanes (many closed experts, equal values, large k) the choices are
// taken one after another.  131072 tokens of 256 float32, top-8: 66 us against 21
// for the bytes, bound by instructions (319 a token, 65% of the issue slots, 52% of
// the pipe of comparisons and integers, with 33% of the warps; 80 registers, for
// which 72 bytes are spilled); by whole warps 76, with a lane's
// experts neighbours, which read every second 16 bytes or fewer at a time, 72,
// one after another 162.  Of 64 experts, top-4, 37 us (warps 56), of 128 bf16,
// top-8, 48 (73).
template <class T, int N, int V, int G>
__global__ void __launch_bounds__(kTeamThreads<V>, kTeamResident<V>)
route_team_kernel(const T *__restrict__ logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                  bool normalize, const uint8_t *__restrict__ mask, RouteOut out, Totals part)
{
    constexpr int kWarps = kTeamThreads<V> / 32, kTeams = kTeamThreads<V> / G;
    constexpr int kSlots = V < 8 ? V : 8;
    __shared__ uint4 s_id[kTeams][kCandidates / 4], s_key[kTeams][kCandidates / 4];
    __shared__ float s_sum[kWarps][G * kSlots];
    __shared__ uint32_t s_count[GC_MAX_EXPERTS];
    __shared__ uint32_t s_warp[kWarps];
    chain_start();
    const uint32_t lane = threadIdx.x & (G - 1), team = threadIdx.x / G, warp = threadIdx.x >> 5, first = lane * N;
    using Row = Logits<T, N, V, G>;
    for (uint32_t e = threadIdx.x; e < experts; e += kTeamThreads<V>) s_count[e] = 0;
    __syncthreads();
    uint32_t *id = reinterpret_cast<uint32_t *>(s_id[team]), *key = reinterpret_cast<uint32_t *>(s_key[team]);
    float sum[V];
    uint32_t routed = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;

    const uint64_t step = uint64_t(gridDim.x) * kTeams;
    Row next;
    auto fetch = [&](uint64_t t) {
        next.load(logits + t * stride, first, experts, t < tokens && (mask == nullptr || mask[t] != 0));
    };
    fetch(uint64_t(blockIdx.x) * kTeams + team);
    // all lanes of a warp go round together, whatever their teams find
    for (uint64_t base = uint64_t(blockIdx.x) * kTeams; base < tokens; base += step) {
        const uint64_t t = base + team;
        const bool inside = t < tokens;
        float x[V], w[V];
        next.values(x);
        fetch(t + step);
        Exponent exponent;
        uint32_t top, left;
        const float total = team_weights<G>(x, w, exponent, top, left);
        const T *row = logits + t * stride;
        int32_t *ids = out.ids + t * topk;
        float *weights = out.weights + t * topk;
        const bool any = total > 0.0f;
        routed += any;
        const float inverse = any ? inverse_of(total) : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = fmaf(w[v], inverse, sum[v]);

        const float least = order_value(max(topk <= G ? kth_largest<G>(left, top, topk) : 0u, kRouteNone + 1));
        using Mask = typename Bits<V>::Type;
        Mask which = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) which |= x[v] >= least ? Mask(1) << v : Mask(0);
        // listed before this lane's: by lanes with one candidate or more, two or more, ...
        const uint32_t mine = Bits<V>::count(which), below = (1u << lane) - 1u;
        uint32_t n = 0, at = 0;
        for (uint32_t more = 0; __any_sync(kRouteFull, mine > more); ++more) {
            const uint32_t have = team_ballot<G>(mine > more);
            n += __popc(have);
            at += __popc(have & below);
        }
        const uint32_t largest_n = __reduce_max_sync(kRouteFull, n);
        if (largest_n <= G) {
            // listed by id; read again, which spares finding them among the registers
            for (; which; which &= which - 1, ++at) id[at] = Row::expert(first, Bits<V>::lowest(which));
            key[lane] = 0;
            __syncwarp();
            uint32_t own = 0, e = 0;
            if (lane < n) {
                e = id[lane];
                own = order_bits(sample_value(row_to_float(row[e])));
                key[lane] = own;
            }
            __syncwarp();
            // before it: the larger ones, and the equal ones of a lower expert
            const uint64_t order = uint64_t(own) << 32 | uint32_t(~e);
            auto before = [&](uint32_t k, uint32_t i) { return uint32_t((uint64_t(k) << 32 | uint32_t(~i)) > order); };
            uint32_t rank = 0;
            for (uint32_t c = 0; c < largest_n; c += 4) {
                const uint4 k = s_key[team][c / 4], i = s_id[team][c / 4];
                rank += before(k.x, i.x) + before(k.y, i.y) + before(k.z, i.z) + before(k.w, i.w);
            }
            const bool chosen = lane < n && rank < topk;
            const float mine_w = chosen ? exponent.weight(order_value(own)) : 0.0f;
            const float scale = normalize ? inverse_of(team_sum<G>(mine_w)) : inverse;
            if (chosen) {
                ids[rank] = int32_t(e);
                weights[rank] = mine_w * scale;
                if (out.counts) atomicAdd(&s_count[e], 1u);
            }
        } else {
            // one after another: a lane's largest with its expert, and which of its logits are left
            Mask rest = ~Mask(0);
            uint32_t whose = 0;
            auto largest_left = [&] {
                left = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t k = order_bits(x[v]);
                    if ((rest >> v & 1u) && k > left) left = k, whose = uint32_t(v);
                }
            };
            largest_left();
            n = 0;
            for (uint32_t j = 0; j < topk; ++j) {
                top = team_max<G>(left);
                // of equal ones the lowest expert
                const uint32_t e = Row::expert(first, 0) + whose / N * (G * N) + whose % N;
                const uint32_t low = ~team_max<G>(left == top ? ~e : 0u);
                if (top <= kRouteNone) continue;
                ++n;
                if (left == top && e == low) {
                    id[j] = e;
                    key[j] = top;
                    rest &= ~(Mask(1) << whose);
                    largest_left();
                }
            }
            __syncwarp();
            float chosen = 0.0f;
            for (uint32_t j = lane; j < n; j += G) chosen += exponent.weight(order_value(key[j]));
            const float scale = normalize ? inverse_of(team_sum<G>(chosen)) : inverse;
            for (uint32_t j = lane; j < n; j += G) {
                ids[j] = int32_t(id[j]);
                weights[j] = exponent.weight(order_value(key[j])) * scale;
                if (out.counts) atomicAdd(&s_count[id[j]], 1u);
            }
        }
        if (inside)
            for (uint32_t j = n + lane; j < topk; j += G) ids[j] = -1, weights[j] = 0.0f;
        __syncwarp();
    }
    if (out.counts == nullptr) return;

    finish<kWarps>(experts, lane == 0 ? routed : 0u, out, part, s_warp, [&](const auto &f) {
        for (int base = 0; base < V; base += kSlots) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v < base || v >= base + kSlots) continue;
                float s = sum[v];
                if (G == 16) s += __shfl_xor_sync(kRouteFull, s, 16);
                if ((threadIdx.x & 31) < G) s_sum[warp][lane * kSlots + (v & (kSlots - 1))] = s;
            }
            __syncthreads();
            const uint32_t v = base + threadIdx.x % kSlots;
            const uint32_t e = threadIdx.x / kSlots * N + v / N * (G * N) + v % N;
            if (threadIdx.x < G * kSlots && e < experts) {
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
        Logits<T, N, V, 1> row;
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

// CTAs: as many as run at a time, each with the tokens of its teams or groups at
// least once; one alone, which spares the second launch, where that has them at
// most kAlone times (of 64 experts 24 tokens 3.3 us, 64 tokens 4.7, by two
// launches 7.2 and 7.0; 128 tokens, four times, 7.1 against 6.7).
constexpr size_t kAlone = 2;

uint32_t grid_of(uint32_t tokens, size_t each, size_t resident)
{
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
    const uint32_t lanes = route_lanes(experts), grid = grid_of(tokens, kGroupThreads / lanes, kGroupResident);
    const Totals part = totals_in(ws, grid, experts);
    route_group_kernel<T, N><<<grid, kGroupThreads, 0, s>>>(static_cast<const T *>(logits), stride, tokens, experts,
                                                            topk, normalize, mask, lanes, out, part);
    return join(part, grid, experts, out, s);
}

template <class T, int N, int V, int G>
cudaError_t run_team(const void *logits, size_t stride, uint32_t tokens, uint32_t experts, uint32_t topk,
                     bool normalize, const uint8_t *mask, const RouteOut &out, uint8_t *ws, cudaStream_t s)
{
    const uint32_t grid = grid_of(tokens, kTeamThreads<V> / G, kTeamResident<V>);
    const Totals part = totals_in(ws, grid, experts);
    route_team_kernel<T, N, V, G><<<grid, kTeamThreads<V>, 0, s>>>(static_cast<const T *>(logits), stride, tokens,
                                                                   experts, topk, normalize, mask, out, part);
    return join(part, grid, experts, out, s);
}

}  // namespace

namespace gch {

size_t expert_route_workspace_bytes(size_t tokens, uint32_t experts)
{
    // whichever kernel the number of choices will take: no more CTAs than this
    const uint32_t n = uint32_t(tokens);
    uint32_t grid;
    if (experts <= kSmallExperts) grid = grid_of(n, kGroupThreads / route_lanes(experts), kGroupResident);
    else if (experts <= 256) grid = grid_of(n, kTeamThreads<16> / 16, kTeamResident<16>);  // 16 tokens, as 512 threads of whole warps
    else grid = grid_of(n, kTeamThreads<64> / 32, kTeamResident<16>);
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
#define GC_ROUTE_CALL_TEAM(T, N, V, G) \
    run_team<T, N, V, G>(logits, stride, tokens, experts, topk, normalize, mask, out, ws, s)
    // more choices than a team of 16 lanes makes
#define GC_ROUTE_WARP(T, whole) \
    if (experts <= 256 && topk > kHalfTopk) GC_ROUTE_TEAM(T, whole, 8, 32, GC_ROUTE_CALL_TEAM)
    GC_ROUTE_BY_DTYPE(dt, experts, whole, GC_ROUTE_CALL, GC_ROUTE_CALL_TEAM, GC_ROUTE_WARP)
}

}  // namespace gch
