// The router of a layer of experts on gfx950: each token's best experts and their weights, how many tokens every expert
// got, the balance loss of both, and the gradient of the logits.
//
// A group of G lanes holds a token's logits in registers, lane l the experts l, l + G, l + 2 G, ..., so they are read
// once: the largest gives the softmax, K rounds of the largest that is left give the choices. Each lane counts its own
// experts' choices and sums their probabilities over all tokens of its workgroup in registers; the workgroups' sums go to
// a workspace and a second kernel adds them in a fixed order, in float64. A single workgroup (few tokens) finishes alone.
#include "gs_types.hpp"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 4096;
constexpr int kBlocks = 1024;      // workgroups of the first kernel, at most
constexpr int64_t kPartials = 1 << 20;  // partial sums of each kind, at most
constexpr int kJoinCols = 64;      // experts of a workgroup of the second kernel
constexpr int kJoinThreads = 1024;
constexpr int kJoinSlices = kJoinThreads / kJoinCols;

// Workgroups for this many tokens with `rows` of them a turn: enough to fill the chip, few enough that their sums are
// soon added.
__host__ inline int route_blocks(int64_t tokens, int rows, int experts) {
    int64_t most = kPartials / experts;
    most = most < kBlocks ? most : kBlocks;
    const int64_t want = (tokens + rows - 1) / rows;
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

// A logit's place in the order of choices: larger first, NaN before all numbers, both zeros alike. 0 is below every
// logit.
__device__ __forceinline__ uint32_t order_of(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kOrderOfNone = 0x007fffffu;  // minus infinity's: an expert that may not be chosen

// The largest of the group's values, and its expert: the lowest among equal ones.
template <int G>
__device__ __forceinline__ void group_best(uint32_t &key, int &expert) {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) {
        const uint32_t k = __shfl_xor(key, d, kWave);
        const int e = __shfl_xor(expert, d, kWave);
        if (k > key || (k == key && e < expert)) {
            key = k;
            expert = e;
        }
    }
}

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t tokens;
    int experts, choices, renormalize;
    int32_t *ids;
    float *weights;
    int32_t *part_counts;  // [workgroups][experts], and the tokens kept [workgroups]
    float *part_shares;
    int32_t *part_kept;
    // of a single workgroup: the results themselves
    int32_t *counts, *kept;
    float *shares, *loss;
};

__device__ __forceinline__ float balance_loss(int experts, double dot, int64_t pairs) {
    return static_cast<float>(experts * dot / static_cast<double>(pairs > 0 ? pairs : 1));
}

template <typename T, int G, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    constexpr int kRows = kThreads / G;
    __shared__ float s_shares[kThreads];
    __shared__ int32_t s_counts[kThreads];
    __shared__ int32_t s_kept[kWaves];
    __shared__ double s_dot[kWaves];
    __shared__ int32_t s_pairs[kWaves];
    const int lane = threadIdx.x % G, group = threadIdx.x / G, E = a.experts, K = a.choices;
    const T *logits = static_cast<const T *>(a.logits);
    // a lane's sums over its tokens, 64 at a time, so that no sum is a long chain of float32 additions
    float share[V], shares[V];
    int32_t count[V], kept = 0, turn = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        share[v] = shares[v] = 0.0f;
        count[v] = 0;
    }
    // all lanes of a wave take as many turns: a token past the end is one that is left out and not written
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < a.tokens;
         first += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t t = first + group;
        const bool there = t < a.tokens;
        const T *row = logits + (there ? t : a.tokens - 1) * E;
        float x[V];
        uint32_t key[V];
        const bool in = there && (!a.mask || a.mask[t] != 0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * G + lane;
            x[v] = e < E ? static_cast<float>(row[e]) : -__builtin_inff();
            key[v] = e < E && in ? order_of(x[v]) : 0u;
        }
        float largest = 0.0f, total = 0.0f, sum = 0.0f;
        bool takes = in;
        for (int k = 0; k < K; ++k) {
            uint32_t best = 0;
            int expert = 0x7fffffff;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] > best) {
                    best = key[v];
                    expert = v * G + lane;
                }
            group_best<G>(best, expert);
            takes = takes && best > kOrderOfNone;
            const uint32_t bits = best & 0x80000000u ? best & 0x7fffffffu : ~best;
            const float value = best == 0xffffffffu ? __builtin_nanf("") : __builtin_bit_cast(float, bits);
            if (k == 0) {
                largest = value;
                float p[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    p[v] = v * G + lane < E ? expf(x[v] - largest) : 0.0f;
                    sum += p[v];
                }
                sum = group_sum<G>(sum);
                if (takes) {
                    const float scale = 1.0f / sum;
#pragma unroll
                    for (int v = 0; v < V; ++v) share[v] = __builtin_fmaf(p[v], scale, share[v]);
                    kept += lane == 0;
                }
            }
            const float e = takes ? expf(value - largest) : 0.0f;
            total += e;
            if (takes) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v * G + lane == expert) {
                        ++count[v];
                        key[v] = 0;
                    }
            }
            if (there && lane == 0) {
                a.ids[t * K + k] = takes ? expert : -1;
                a.weights[t * K + k] = takes ? a.renormalize ? e : e / sum : 0.0f;
            }
        }
        if (++turn % 64 == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                shares[v] += share[v];
                share[v] = 0.0f;
            }
        }
        // read back by the lane that wrote them
        if (a.renormalize && in && there && lane == 0 && total != 0.0f)
            for (int k = 0; k < K; ++k) a.weights[t * K + k] /= total;
    }
    // the workgroup's sums: its groups' in order
    const bool alone = gridDim.x == 1;
    double dot = 0.0;
    int32_t pairs = 0;
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) kept += __shfl_xor(kept, d, kWave);
    if (threadIdx.x % kWave == 0) s_kept[threadIdx.x / kWave] = kept;
    __syncthreads();
    kept = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) kept += s_kept[w];
    const float inverse = 1.0f / static_cast<float>(kept > 0 ? kept : 1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        __syncthreads();
        s_shares[threadIdx.x] = shares[v] + share[v];
        s_counts[threadIdx.x] = count[v];
        __syncthreads();
        for (int l = threadIdx.x; l < G; l += kThreads) {
            const int e = v * G + l;
            if (e >= E) continue;
            float s = 0.0f;
            int32_t c = 0;
            for (int r = 0; r < kRows; ++r) {
                s += s_shares[r * G + l];
                c += s_counts[r * G + l];
            }
            if (alone) {
                s *= inverse;
                a.shares[e] = s;
                a.counts[e] = c;
                dot += static_cast<double>(s) * c;
                pairs += c;
            } else {
                a.part_shares[static_cast<int64_t>(blockIdx.x) * E + e] = s;
                a.part_counts[static_cast<int64_t>(blockIdx.x) * E + e] = c;
            }
        }
    }
    if (!alone) {
        if (threadIdx.x == 0) a.part_kept[blockIdx.x] = kept;
        return;
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) {
        dot += __shfl_xor(dot, d, kWave);
        pairs += __shfl_xor(pairs, d, kWave);
    }
    if (threadIdx.x % kWave == 0) {
        s_dot[threadIdx.x / kWave] = dot;
        s_pairs[threadIdx.x / kWave] = pairs;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = 0.0;
        int64_t n = 0;
        for (int w = 0; w < kWaves; ++w) {
            dot += s_dot[w];
            n += s_pairs[w];
        }
        *a.loss = balance_loss(E, dot, n);
        *a.kept = kept;
    }
}

// Sum of v over the workgroup's threads in a fixed order, in every thread.
template <int THREADS, typename S>
__device__ __forceinline__ S workgroup_sum(S v, S *slots) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    __syncthreads();
    if (threadIdx.x % kWave == 0) slots[threadIdx.x / kWave] = v;
    __syncthreads();
    S s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) s += slots[w];
    return s;
}

// Adds the workgroups' sums of kJoinCols experts; where that is all of them, the loss too.
__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(const int32_t *__restrict__ part_counts,
                                                                  const float *__restrict__ part_shares,
                                                                  const int32_t *__restrict__ part_kept, int parts,
                                                                  int experts, int32_t *__restrict__ counts,
                                                                  float *__restrict__ shares,
                                                                  int32_t *__restrict__ kept_out,
                                                                  float *__restrict__ loss) {
    __shared__ double s_share[kJoinThreads];
    __shared__ int32_t s_count[kJoinThreads];
    __shared__ double s_dot[kJoinThreads / kWave];
    __shared__ int32_t s_sum[kJoinThreads / kWave];
    int32_t kept = 0;
    for (int b = threadIdx.x; b < parts; b += kJoinThreads) kept += part_kept[b];
    kept = workgroup_sum<kJoinThreads>(kept, s_sum);
    const int col = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols, e = blockIdx.x * kJoinCols + col;
    double s = 0.0;
    int32_t c = 0;
    if (e < experts)
        for (int b = slice; b < parts; b += kJoinSlices) {
            s += static_cast<double>(part_shares[static_cast<int64_t>(b) * experts + e]);
            c += part_counts[static_cast<int64_t>(b) * experts + e];
        }
    s_share[threadIdx.x] = s;
    s_count[threadIdx.x] = c;
    __syncthreads();
    double dot = 0.0;
    int32_t pairs = 0;
    if (slice == 0 && e < experts) {
        for (int i = 1; i < kJoinSlices; ++i) {
            s += s_share[i * kJoinCols + col];
            c += s_count[i * kJoinCols + col];
        }
        s /= kept > 0 ? kept : 1;
        shares[e] = static_cast<float>(s);
        counts[e] = c;
        dot = s * c;
        pairs = c;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *kept_out = kept;
    if (gridDim.x > 1) return;
    dot = workgroup_sum<kJoinThreads>(dot, s_dot);
    pairs = workgroup_sum<kJoinThreads>(pairs, s_sum);
    if (threadIdx.x == 0) *loss = balance_loss(experts, dot, pairs);
}

__global__ __launch_bounds__(kJoinThreads) void route_loss_kernel(const int32_t *__restrict__ counts,
                                                                  const float *__restrict__ shares, int experts,
                                                                  float *__restrict__ loss) {
    __shared__ double s_dot[kJoinThreads / kWave];
    __shared__ int32_t s_sum[kJoinThreads / kWave];
    double dot = 0.0;
    int32_t pairs = 0;
    for (int e = threadIdx.x; e < experts; e += kJoinThreads) {
        dot += static_cast<double>(shares[e]) * counts[e];
        pairs += counts[e];
    }
    dot = workgroup_sum<kJoinThreads>(dot, s_dot);
    pairs = workgroup_sum<kJoinThreads>(pairs, s_sum);
    if (threadIdx.x == 0) *loss = balance_loss(experts, dot, pairs);
}

// With nothing to route: counts, shares and the loss are zeros.
__global__ __launch_bounds__(kThreads) void route_none_kernel(int experts, int32_t *counts, float *shares,
                                                              int32_t *kept, float *loss) {
    for (int e = threadIdx.x; e < experts; e += kThreads) {
        counts[e] = 0;
        shares[e] = 0.0f;
    }
    if (threadIdx.x == 0) {
        *kept = 0;
        *loss = 0.0f;
    }
}

struct RouteBwdArgs {
    const void *logits;
    const int32_t *ids, *counts, *kept;
    const float *weights, *grad_weights, *grad_loss;
    int64_t tokens;
    int experts, choices, renormalize;
    void *grad_logits;
};

// The gradient of a token's logits, formed again from them:
//   through the weights  [j = ids_k] w_k (g_k - sum_i g_i w_i), or, not renormalised, the sum's part times p_j,
//   through the loss     grad_loss * experts / kept * p_j (f_j - sum_e f_e p_e),  f_e = counts_e / sum of counts.
template <typename T, int G, int V>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdArgs a) {
    constexpr int kRows = kThreads / G;
    __shared__ int32_t s_sum[kWaves];
    const int lane = threadIdx.x % G, group = threadIdx.x / G, E = a.experts, K = a.choices;
    float f[V], scale = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.0f;
    if (a.grad_loss) {
        int32_t pairs = 0;
        for (int e = threadIdx.x; e < E; e += kThreads) pairs += a.counts[e];
        pairs = workgroup_sum<kThreads>(pairs, s_sum);
        const int32_t kept = *a.kept;
        scale = *a.grad_loss * static_cast<float>(E) / static_cast<float>(kept > 0 ? kept : 1);
        const float inverse = 1.0f / static_cast<float>(pairs > 0 ? pairs : 1);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * G + lane < E) f[v] = static_cast<float>(a.counts[v * G + lane]) * inverse;
    }
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < a.tokens;
         first += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t t = first + group;
        const bool there = t < a.tokens;
        const int64_t at = there ? t : a.tokens - 1;
        const T *row = static_cast<const T *>(a.logits) + at * E;
        const int32_t *ids = a.ids + at * K;
        const bool in = ids[0] >= 0;
        float p[V], most = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = v * G + lane < E ? static_cast<float>(row[v * G + lane]) : -__builtin_inff();
            most = fmaxf(most, p[v]);
        }
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d, kWave));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = v * G + lane < E ? expf(p[v] - most) : 0.0f;
            sum += p[v];
        }
        const float inverse = 1.0f / group_sum<G>(sum);
        float mean = 0.0f, total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] *= inverse;
            mean = __builtin_fmaf(p[v], f[v], mean);
        }
        mean = group_sum<G>(mean);
        if (a.grad_weights)
            for (int k = 0; k < K; ++k)
                if (ids[k] >= 0) total = __builtin_fmaf(a.grad_weights[at * K + k], a.weights[at * K + k], total);
        float g[V];
        const float through = a.renormalize ? 0.0f : total;
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = p[v] * __builtin_fmaf(scale, f[v] - mean, -through);
        if (a.grad_weights)
            for (int k = 0; k < K; ++k) {
                const int e = ids[k];
                if (e < 0) continue;
                const float w = a.weights[at * K + k], gw = a.grad_weights[at * K + k];
                const float add = a.renormalize ? w * (gw - total) : w * gw;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v * G + lane == e) g[v] += add;
            }
        if (there) {
            T *out = static_cast<T *>(a.grad_logits) + t * E;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * G + lane < E) out[v * G + lane] = static_cast<T>(in ? g[v] : 0.0f);
        }
    }
}

constexpr int64_t kLimit = int64_t(1) << 31;

gs_status check_route(const char *name, int64_t tokens, int experts, int64_t choices, int dtype) {
    if (tokens < 0 || tokens >= kLimit || choices < 1 || choices >= kLimit || tokens * choices >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "%s: need tokens >= 0, choices >= 1 and tokens * choices < 2^31", name);
    if (experts < 1 || experts > kMaxExperts)
        return fail(GS_ERR_INVALID_ARG, "%s: experts = %d outside [1, %d]", name, experts, kMaxExperts);
    if (choices > experts)
        return fail(GS_ERR_INVALID_ARG, "%s: choices = %lld above experts = %d", name,
                    static_cast<long long>(choices), experts);
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "%s: dtype = %d is no gs_dtype", name, dtype);
    return GS_OK;
}

// Lanes that share a token: as many as it has experts, up to a wave.
inline int route_lanes(int experts) {
    int g = 1;
    while (g < experts && g < kWave) g *= 2;
    return g;
}

struct RouteRoom {
    int blocks;
    size_t bytes, counts, shares, kept;
};
RouteRoom route_room(int64_t tokens, int experts) {
    RouteRoom r;
    r.blocks = route_blocks(tokens, kThreads / route_lanes(experts), experts);
    const size_t n = static_cast<size_t>(r.blocks) * experts * 4;
    r.counts = 0;
    r.shares = align_up(n, 256);
    r.kept = r.shares + align_up(n, 256);
    r.bytes = r.blocks == 1 ? 0 : r.kept + align_up(static_cast<size_t>(r.blocks) * 4, 256);
    return r;
}

}  // namespace
}  // namespace gs

using namespace gs;

// Launches kernel<T, G, V> for the type code and the number of experts.
#define GS_ROUTE_LAUNCH_GV(kernel, T, G, V) \
    hipLaunchKernelGGL((kernel<T, G, V>), grid, dim3(kThreads), 0, stream, a)
#define GS_ROUTE_LAUNCH_T(kernel, T)                                    \
    do {                                                                \
        if (experts <= 1) GS_ROUTE_LAUNCH_GV(kernel, T, 1, 1);          \
        else if (experts <= 2) GS_ROUTE_LAUNCH_GV(kernel, T, 2, 1);     \
        else if (experts <= 4) GS_ROUTE_LAUNCH_GV(kernel, T, 4, 1);     \
        else if (experts <= 8) GS_ROUTE_LAUNCH_GV(kernel, T, 8, 1);     \
        else if (experts <= 16) GS_ROUTE_LAUNCH_GV(kernel, T, 16, 1);   \
        else if (experts <= 32) GS_ROUTE_LAUNCH_GV(kernel, T, 32, 1);   \
        else if (experts <= 64) GS_ROUTE_LAUNCH_GV(kernel, T, 64, 1);   \
        else if (experts <= 128) GS_ROUTE_LAUNCH_GV(kernel, T, 64, 2);  \
        else if (experts <= 256) GS_ROUTE_LAUNCH_GV(kernel, T, 64, 4);  \
        else if (experts <= 1024) GS_ROUTE_LAUNCH_GV(kernel, T, 64, 16); \
        else GS_ROUTE_LAUNCH_GV(kernel, T, 64, 64);                     \
        GS_LAUNCH_TRY(#kernel);                                         \
    } while (0)
#define GS_ROUTE_LAUNCH(kernel)                                   \
    do {                                                          \
        if (dtype == GS_F32) GS_ROUTE_LAUNCH_T(kernel, float);    \
        else if (dtype == GS_BF16) GS_ROUTE_LAUNCH_T(kernel, __bf16); \
        else GS_ROUTE_LAUNCH_T(kernel, _Float16);                 \
    } while (0)

extern "C" size_t gs_expert_route_workspace_bytes(int64_t tokens, int experts) {
    if (tokens < 0 || tokens >= kLimit || experts < 1 || experts > kMaxExperts) return 0;
    return route_room(tokens, experts).bytes;
}

extern "C" gs_status gs_expert_route(const void *logits, const uint8_t *mask, int64_t tokens, int experts,
                                     int64_t choices, int renormalize, int dtype, int32_t *ids, float *weights,
                                     int32_t *counts, float *shares, float *loss, int32_t *kept, void *workspace,
                                     size_t workspace_bytes, void *stream_handle) {
    const gs_status bad = check_route("gs_expert_route", tokens, experts, choices, dtype);
    if (bad != GS_OK) return bad;
    if (!counts || !shares || !loss || !kept || (tokens > 0 && (!logits || !ids || !weights)))
        return fail(GS_ERR_INVALID_ARG, "gs_expert_route: a required pointer is NULL");
    const RouteRoom room = route_room(tokens, experts);
    if (room.bytes > 0 && (!workspace || workspace_bytes < room.bytes))
        return fail(GS_ERR_WORKSPACE, "gs_expert_route: need %zu workspace bytes, got %zu", room.bytes,
                    workspace ? workspace_bytes : 0);
    const size_t pairs = static_cast<size_t>(tokens) * choices, n = static_cast<size_t>(experts);
    const gs_status over = check_apart("gs_expert_route",
                                       {{"ids", ids, pairs * 4}, {"weights", weights, pairs * 4},
                                        {"counts", counts, n * 4}, {"shares", shares, n * 4}, {"loss", loss, 4},
                                        {"kept", kept, 4}, {"workspace", workspace, room.bytes}},
                                       {{"logits", logits, static_cast<size_t>(tokens) * n * dtype_size(dtype)},
                                        {"mask", mask, static_cast<size_t>(tokens)}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    if (tokens == 0) {
        hipLaunchKernelGGL(route_none_kernel, dim3(1), dim3(kThreads), 0, stream, experts, counts, shares, kept, loss);
        GS_LAUNCH_TRY("route_none_kernel");
        return ok();
    }
    char *at = static_cast<char *>(workspace);
    RouteArgs a = {logits, mask, tokens, experts, static_cast<int>(choices), renormalize ? 1 : 0, ids, weights};
    if (room.bytes > 0) {
        a.part_counts = reinterpret_cast<int32_t *>(at + room.counts);
        a.part_shares = reinterpret_cast<float *>(at + room.shares);
        a.part_kept = reinterpret_cast<int32_t *>(at + room.kept);
    }
    a.counts = counts;
    a.kept = kept;
    a.shares = shares;
    a.loss = loss;
    const dim3 grid(static_cast<unsigned>(room.blocks));
    GS_ROUTE_LAUNCH(route_kernel);
    if (room.blocks == 1) return ok();
    const int joins = (experts + kJoinCols - 1) / kJoinCols;
    hipLaunchKernelGGL(route_join_kernel, dim3(static_cast<unsigned>(joins)), dim3(kJoinThreads), 0, stream,
                       a.part_counts, a.part_shares, a.part_kept, room.blocks, experts, counts, shares, kept, loss);
    GS_LAUNCH_TRY("route_join_kernel");
    if (joins > 1) {
        hipLaunchKernelGGL(route_loss_kernel, dim3(1), dim3(kJoinThreads), 0, stream, counts, shares, experts, loss);
        GS_LAUNCH_TRY("route_loss_kernel");
    }
    return ok();
}

extern "C" gs_status gs_expert_route_bwd(const void *logits, const int32_t *ids, const float *weights,
                                         const int32_t *counts, const int32_t *kept, const float *grad_weights,
                                         const float *grad_loss, int64_t tokens, int experts, int64_t choices,
                                         int renormalize, int dtype, void *grad_logits, void *stream_handle) {
    const gs_status bad = check_route("gs_expert_route_bwd", tokens, experts, choices, dtype);
    if (bad != GS_OK) return bad;
    if (tokens == 0) return ok();
    if (!logits || !ids || !weights || !counts || !kept || !grad_logits)
        return fail(GS_ERR_INVALID_ARG, "gs_expert_route_bwd: a required pointer is NULL");
    const size_t pairs = static_cast<size_t>(tokens) * choices, n = static_cast<size_t>(experts);
    const size_t bytes = static_cast<size_t>(tokens) * n * dtype_size(dtype);
    const gs_status over = check_apart("gs_expert_route_bwd", {{"grad_logits", grad_logits, bytes}},
                                       {{"logits", logits, bytes}, {"ids", ids, pairs * 4},
                                        {"weights", weights, pairs * 4}, {"counts", counts, n * 4}, {"kept", kept, 4},
                                        {"grad_weights", grad_weights, pairs * 4}, {"grad_loss", grad_loss, 4}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    RouteBwdArgs a = {logits, ids, counts, kept, weights, grad_weights, grad_loss, tokens, experts,
                      static_cast<int>(choices), renormalize ? 1 : 0, grad_logits};
    const int64_t rows = kThreads / route_lanes(experts), want = (tokens + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>(want < 8 * kBlocks ? want : 8 * kBlocks));
    GS_ROUTE_LAUNCH(route_bwd_kernel);
    return ok();
}
