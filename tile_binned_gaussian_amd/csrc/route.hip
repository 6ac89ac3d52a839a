// The router of a layer of experts on gfx950: each token's best experts and their weights, how many tokens every expert
// got, the balance loss of both, and the gradient of the logits.
//
// A group of G lanes holds a token's logits in registers, lane l the experts l V to l V + V - 1, so they are read once:
// the largest gives the softmax, K rounds of the largest that is left give the choices. Each lane counts its own
// experts' choices and sums their probabilities over all tokens of its workgroup in registers; the workgroups' sums go to
// a workspace and a second kernel adds them in a fixed order, in float64. A single workgroup (few tokens) finishes alone.
//
// 1000000 x 8 float32, 2 choices: 19.5 us (2.5 TB/s: a token a lane, so rounds of comparisons, exponentials and stores of
// 8 bytes a token fill the time) and 5.1 for the second kernel; the gradient of 32768 x 64, 8 choices 8.7 us (2.3 TB/s).
// Eight lanes a token instead took 99 us with the second kernel, 64 lanes the gradient 30: values crossed lanes by LDS.
#include <type_traits>

#include "gs_types.hpp"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 4096;
constexpr int kBlocks = 1024;      // workgroups of the first kernel, at most
constexpr int64_t kPartials = 1 << 20;  // partial sums of each kind, at most
constexpr int kJoinCols = 64;      // experts of a workgroup of the second kernel, at most
constexpr int kJoinThreads = 1024;

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

// The value of the lane that differs in one bit of its number, or in a whole run of them: once the lanes of each half
// agree, any of the other half will do, and within 16 lanes the mirrored one costs no LDS instruction.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t v) {
    if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
    else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
    else if constexpr (D == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
    else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
    else return __shfl_xor(v, D, kWave);
}
// Folds f over the group's lanes, from neighbours on: every lane gets the same.
template <int G, int D = 1, typename F>
__device__ __forceinline__ void fold(const F &f) {
    if constexpr (D < G) {
        f(std::integral_constant<int, D>());
        fold<G, D * 2>(f);
    }
}
template <int G>
__device__ __forceinline__ float sum_of(float v) {
    fold<G>([&](auto d) {
        v += __builtin_bit_cast(float, across<decltype(d)::value>(__builtin_bit_cast(uint32_t, v)));
    });
    return v;
}

// The largest of the group's values, and its expert: the lowest among equal ones.
template <int G>
__device__ __forceinline__ void group_best(uint32_t &key, uint32_t &expert) {
    fold<G>([&](auto d) {
        const uint32_t k = across<decltype(d)::value>(key), e = across<decltype(d)::value>(expert);
        const bool take = k > key || (k == key && e < expert);
        key = take ? k : key;
        expert = take ? e : expert;
    });
}

// Lane l of the group has experts l * V to l * V + V - 1. WHOLE: there are G * V of them.
template <int G, int V, bool WHOLE, typename T>
__device__ __forceinline__ void load_row(const T *row, int lane, int experts, float (&x)[V]) {
    if constexpr (WHOLE) {
        typedef T P __attribute__((ext_vector_type(V)));
        typedef P U __attribute__((aligned(sizeof(T))));
        const P p = *reinterpret_cast<const U *>(row + lane * V);
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = static_cast<float>(p[v]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            x[v] = static_cast<float>(row[e < experts ? e : experts - 1]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = lane * V + v < experts ? x[v] : -__builtin_inff();
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

template <typename T, int G, int V, bool WHOLE>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    constexpr int kRows = kThreads / G;
    constexpr int kHold = G == 1 ? 4 : 1;  // choices that a lane holds until their sum is known
    __shared__ float s_shares[kWaves][G * V];
    __shared__ int32_t s_counts[kWaves][G * V];
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
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + group;
    float next[V];
    uint8_t next_in = 1;
    const auto fetch = [&](int64_t at) {
        at = at < a.tokens ? at : a.tokens - 1;
        load_row<G, V, WHOLE>(logits + at * E, lane, E, next);
        if (a.mask) next_in = a.mask[at];
    };
    fetch(t);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < a.tokens; first += step, t += step) {
        const bool there = t < a.tokens, in = there && next_in != 0;
        float x[V];
        uint32_t key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = next[v];
            key[v] = in ? order_of(x[v]) : 0u;
            if (!WHOLE && lane * V + v >= E) key[v] = 0u;
        }
        if (first + step < a.tokens) fetch(t + step);
        float largest = 0.0f, total = 0.0f, sum = 0.0f;
        bool takes = in;
        int32_t my_id[kHold];
        float my_e[kHold];
        const bool held = K <= G * kHold;
        const auto choose = [&](int k, int slot) {
            uint32_t best = key[0], expert = static_cast<uint32_t>(lane * V);
#pragma unroll
            for (int v = 1; v < V; ++v) {
                const bool take = key[v] > best;
                best = take ? key[v] : best;
                expert = take ? static_cast<uint32_t>(lane * V + v) : expert;
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
                    p[v] = expf(x[v] - largest);  // 0 past the last expert
                    if (!WHOLE && lane * V + v >= E) p[v] = 0.0f;
                    sum += p[v];
                }
                sum = sum_of<G>(sum);
                const float scale = takes ? 1.0f / sum : 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) share[v] = takes ? __builtin_fmaf(p[v], scale, share[v]) : share[v];
                kept += takes && lane == 0;
            }
            const float e = takes ? expf(value - largest) : 0.0f;
            total += e;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool mine = takes && static_cast<uint32_t>(lane * V + v) == expert;
                count[v] += mine;
                key[v] = mine ? 0u : key[v];
            }
            const int32_t id = takes ? static_cast<int32_t>(expert) : -1;
            if (held) {
                if (G == 1 || k == lane) {
                    my_id[slot] = id;
                    my_e[slot] = e;
                }
            } else if (there && lane == 0) {
                a.ids[t * K + k] = id;
                a.weights[t * K + k] = e;
            }
        };
        if constexpr (G == 1) {
#pragma unroll
            for (int k = 0; k < kHold; ++k)
                if (k < K) choose(k, k);
            for (int k = kHold; k < K; ++k) choose(k, 0);
        } else {
            for (int k = 0; k < K; ++k) choose(k, 0);
        }
        // divided by the sum of the chosen or of all: no token has an empty sum but one that is left out
        const float divisor = a.renormalize ? total : sum;
        if (held) {
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const int k = G == 1 ? i : lane;
                if (there && k < K) {
                    a.ids[t * K + k] = my_id[i];
                    a.weights[t * K + k] = my_id[i] >= 0 ? my_e[i] / divisor : 0.0f;
                }
            }
        } else if (there && lane == 0) {  // read back by the lane that wrote them
            for (int k = 0; k < K; ++k)
                a.weights[t * K + k] = a.ids[t * K + k] >= 0 ? a.weights[t * K + k] / divisor : 0.0f;
        }
        if (++turn % 64 == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                shares[v] += share[v];
                share[v] = 0.0f;
            }
        }
    }
    // the workgroup's sums: over the wave's groups, then the waves in order
    const bool alone = gridDim.x == 1;
    const int wave = threadIdx.x / kWave;
    double dot = 0.0;
    int32_t pairs = 0;
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) kept += __shfl_xor(kept, d, kWave);
    if (threadIdx.x % kWave == 0) s_kept[wave] = kept;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = shares[v] + share[v];
        int32_t c = count[v];
#pragma unroll
        for (int d = G; d < kWave; d <<= 1) {
            s += __shfl_xor(s, d, kWave);
            c += __shfl_xor(c, d, kWave);
        }
        if (threadIdx.x % kWave < G) {
            s_shares[wave][lane * V + v] = s;
            s_counts[wave][lane * V + v] = c;
        }
    }
    __syncthreads();
    kept = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) kept += s_kept[w];
    const float inverse = 1.0f / static_cast<float>(kept > 0 ? kept : 1);
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float s = 0.0f;
        int32_t c = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            s += s_shares[w][e];
            c += s_counts[w][e];
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

// Adds the workgroups' sums of `cols` experts (a power of two); where that is all of them, the loss too. The threads of an
// expert share its sums and are added pair by pair.
__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(const int32_t *__restrict__ part_counts,
                                                                  const float *__restrict__ part_shares,
                                                                  const int32_t *__restrict__ part_kept, int parts,
                                                                  int experts, int cols, int32_t *__restrict__ counts,
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
    const int col = threadIdx.x % cols, slice = threadIdx.x / cols, slices = kJoinThreads / cols;
    const int e = blockIdx.x * cols + col;
    double s = 0.0;
    int32_t c = 0;
    if (e < experts)
#pragma unroll 4
        for (int b = slice; b < parts; b += slices) {
            s += static_cast<double>(part_shares[static_cast<int64_t>(b) * experts + e]);
            c += part_counts[static_cast<int64_t>(b) * experts + e];
        }
    s_share[threadIdx.x] = s;
    s_count[threadIdx.x] = c;
    for (int n = slices / 2; n > 0; n >>= 1) {
        __syncthreads();
        if (slice < n) {
            s_share[threadIdx.x] = s += s_share[threadIdx.x + n * cols];
            s_count[threadIdx.x] = c += s_count[threadIdx.x + n * cols];
        }
    }
    double dot = 0.0;
    int32_t pairs = 0;
    if (slice == 0 && e < experts) {
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
// Lane k of the group has the token's choice k (and k + G, ...), and gives it to the others in turn.
template <typename T, int G, int V, bool WHOLE>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdArgs a) {
    constexpr int kRows = kThreads / G;
    __shared__ int32_t s_sum[kWaves];
    const int lane = threadIdx.x % G, group = threadIdx.x / G, E = a.experts, K = a.choices;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + group;
    struct Choice {
        int32_t id;
        float w, g;
    };
    float next[V];
    Choice next_choice;
    const auto choice = [&](int64_t at, int k) {
        const int64_t i = at * K + (k < K ? k : K - 1);
        Choice c = {a.ids[i], a.weights[i], 0.0f};
        if (a.grad_weights) c.g = a.grad_weights[i];
        if (k >= K) c.id = -1;
        return c;
    };
    const auto fetch = [&](int64_t at) {
        at = at < a.tokens ? at : a.tokens - 1;
        load_row<G, V, WHOLE>(static_cast<const T *>(a.logits) + at * E, lane, E, next);
        next_choice = choice(at, G == 1 ? 0 : lane);
    };
    fetch(t);
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
            if (lane * V + v < E) f[v] = static_cast<float>(a.counts[lane * V + v]) * inverse;
    }
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < a.tokens; first += step, t += step) {
        const bool there = t < a.tokens;
        const int64_t at = there ? t : a.tokens - 1;
        float p[V], most = -__builtin_inff(), sum = 0.0f;
        const Choice mine = next_choice;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = next[v];
            most = fmaxf(most, p[v]);
        }
        if (first + step < a.tokens) fetch(t + step);
        fold<G>([&](auto d) {
            most = fmaxf(most, __builtin_bit_cast(float, across<decltype(d)::value>(__builtin_bit_cast(uint32_t, most))));
        });
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = expf(p[v] - most);
            if (!WHOLE && lane * V + v >= E) p[v] = 0.0f;
            sum += p[v];
        }
        const float inverse = 1.0f / sum_of<G>(sum);
        float mean = 0.0f, total = mine.id >= 0 ? mine.g * mine.w : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] *= inverse;
            mean = __builtin_fmaf(p[v], f[v], mean);
        }
        mean = sum_of<G>(mean);
        for (int k = G; k < K; k += G) {
            const Choice c = choice(at, k + lane);
            total += c.id >= 0 ? c.g * c.w : 0.0f;
        }
        total = sum_of<G>(total);
        // a token that was left out has no first choice
        const bool in = __shfl(mine.id, threadIdx.x % kWave - lane, kWave) >= 0;
        float g[V];
        const float through = a.renormalize ? 0.0f : total;
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = p[v] * __builtin_fmaf(scale, f[v] - mean, -through);
        const auto add = [&](const Choice &c, int from) {
            const float part = a.renormalize ? c.w * (c.g - total) : c.w * c.g;
            const int32_t id = G == 1 ? c.id : __shfl(c.id, threadIdx.x % kWave - lane + from, kWave);
            const float of = G == 1 ? part : __shfl(part, threadIdx.x % kWave - lane + from, kWave);
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] += id == lane * V + v ? of : 0.0f;
        };
        for (int k = 0; k < K && k < G; ++k) add(mine, k);
        for (int k = G; k < K; k += G) {
            const Choice c = choice(at, k + lane);
            for (int i = 0; i < G && k + i < K; ++i) add(c, i);
        }
        T *out = static_cast<T *>(a.grad_logits) + at * E;
        if (!there) continue;
        if constexpr (WHOLE) {
            typedef T P __attribute__((ext_vector_type(V)));
            typedef P U __attribute__((aligned(sizeof(T))));
            P o;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = static_cast<T>(in ? g[v] : 0.0f);
            *reinterpret_cast<U *>(out + lane * V) = o;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (lane * V + v < E) out[lane * V + v] = static_cast<T>(in ? g[v] : 0.0f);
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

// Lanes that share a token, and a lane's experts. Up to 16 experts a lane has a token of its own and no value crosses
// lanes; up to 256 they are 16 lanes, within which values cross without LDS. Float32, 2 choices, forward / gradient in us:
//   1000000 x 8    one lane 24 / 19, eight 56 / 28           300000 x 64   16 lanes 55 / 31, eight 43 / 30, 64 162 / 68
//   1000000 x 16   one lane 37 / 36, eight 61 / 34           200000 x 128  16 lanes 56 / 40, eight 57 / 47, 64 123 / 56
//   500000 x 32    eight lanes 44 / 25, one 50 / 38,         100000 x 256  16 lanes 57 / 52, eight 90 / 68, 64 79 / 40
//                  16 66 / 35                                20000 x 1024  64 lanes 67 / 130
// A number of experts that fills no lane's load costs more: 12 for 16 46 / 57, 100 for 128 65 / 73, 200 for 256 76 / 117.
// Each further choice is a round: 8 of 8 79 / 92, 8 of 64 121 / 38, 8 of 256 99 / 55. The largest lane, 64 experts of more
// than 1024, leaves 226 registers to scratch.
constexpr int route_lanes(int experts) { return experts <= 16 ? 1 : experts <= 32 ? 8 : experts <= 256 ? 16 : 64; }
constexpr int route_columns(int experts) {
    return experts <= 4 ? 4 : experts <= 8 ? 8 : experts <= 16 ? 16 : experts <= 64 ? 4 : experts <= 128 ? 8
           : experts <= 1024 ? 16 : 64;
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

// Launches kernel<T, G, V, WHOLE> for the type code and the number of experts.
#define GS_ROUTE_LAUNCH_V(kernel, T, MOST, WHOLE)                                                              \
    hipLaunchKernelGGL((kernel<T, route_lanes(MOST), route_columns(MOST), WHOLE>), grid, dim3(kThreads), 0, stream, a)
#define GS_ROUTE_LAUNCH_W(kernel, T, MOST)                                 \
    do {                                                                   \
        if (experts == MOST) GS_ROUTE_LAUNCH_V(kernel, T, MOST, true);     \
        else GS_ROUTE_LAUNCH_V(kernel, T, MOST, false);                    \
    } while (0)
#define GS_ROUTE_LAUNCH_T(kernel, T)                                \
    do {                                                            \
        if (experts <= 4) GS_ROUTE_LAUNCH_W(kernel, T, 4);          \
        else if (experts <= 8) GS_ROUTE_LAUNCH_W(kernel, T, 8);     \
        else if (experts <= 16) GS_ROUTE_LAUNCH_W(kernel, T, 16);   \
        else if (experts <= 32) GS_ROUTE_LAUNCH_W(kernel, T, 32);   \
        else if (experts <= 64) GS_ROUTE_LAUNCH_W(kernel, T, 64);   \
        else if (experts <= 128) GS_ROUTE_LAUNCH_W(kernel, T, 128); \
        else if (experts <= 256) GS_ROUTE_LAUNCH_W(kernel, T, 256); \
        else if (experts <= 1024) GS_ROUTE_LAUNCH_V(kernel, T, 1024, false); \
        else GS_ROUTE_LAUNCH_V(kernel, T, 4096, false);             \
        GS_LAUNCH_TRY(#kernel);                                     \
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
    int cols = 1;
    while (cols < experts && cols < kJoinCols) cols *= 2;
    const int joins = (experts + cols - 1) / cols;
    hipLaunchKernelGGL(route_join_kernel, dim3(static_cast<unsigned>(joins)), dim3(kJoinThreads), 0, stream,
                       a.part_counts, a.part_shares, a.part_kept, room.blocks, experts, cols, counts, shares, kept, loss);
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
    const dim3 grid(static_cast<unsigned>(want < 2 * kBlocks ? want : 2 * kBlocks));
    GS_ROUTE_LAUNCH(route_bwd_kernel);
    return ok();
}
