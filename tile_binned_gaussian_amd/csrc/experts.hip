// Tokens sorted by expert and back on gfx950: the plan (a stable counting sort of the (token, choice) pairs by
// expert), the copy of token rows into sorted order, and their weighted sum back with its gradient.
//
// Every row operation walks the tokens, not the sorted rows: a token's own row (x in the dispatch, the output
// gradient in the combine's backward) is read once for all of its choices, and the sorted rows, which are the bulk of
// the bytes, are each read or written once. No atomics on memory: results do not depend on the order of workgroups.
//
// All of it is bound by memory. 32768 tokens, 8 choices of 64 experts, rows of 2048 bf16 (2.4 GB): plan 13 us, dispatch
// 231 us (5.2 TB/s), combine 205 us (5.9 TB/s, near what plain reads reach); 16384 x 2 rows of 4096 bf16: combine's
// backward 128 us (5.1 TB/s). A large copy runs at 4.8 TB/s. Few tokens are three launches of 3 to 4 us each.
#include "gs_types.hpp"

namespace gs {
namespace {

// ------------------------------------------------------------------------------------------------------------
// the plan

constexpr int kMaxExperts = 4096;
constexpr int kPlanThreads = 1024;   // up to kWideExperts experts
constexpr int kWideThreads = 256;    // above: one LDS counter per expert and wave has to fit
constexpr int kWideExperts = 1024;
// LDS of expert_place_kernel: a counter for every wave and two more for every expert. The most is the kernel's attribute,
// whatever a call needs, so that calls from several host threads set one value.
constexpr size_t plan_lds(int threads, int experts) {
    return static_cast<size_t>(threads / kWave + 2) * static_cast<size_t>(experts) * sizeof(int32_t);
}
constexpr size_t kPlanLds = plan_lds(kWideThreads, kMaxExperts);
static_assert(kPlanLds >= plan_lds(kPlanThreads, kWideExperts) && kPlanLds <= 159 * 1024, "both fit");
// Pairs that one workgroup takes alone, in one launch: 4096 pairs of 8 to 256 experts 7.1 to 8.8 us in one launch and 7.3
// to 7.9 in two, whose second costs the host 3.5 us more; 8192 pairs 10.4 to 13.4 us alone, 8.4 to 9.1 in two.
constexpr int64_t kPlanAlone = 4096;
constexpr int64_t kPlanChunks = 256;  // workgroups, at most

// Pairs of a workgroup: one step of its threads, or what 256 workgroups need.
int64_t plan_chunk(int64_t pairs) {
    if (pairs <= kPlanAlone) return kPlanAlone;
    const int64_t c = (pairs + kPlanChunks - 1) / kPlanChunks;
    return (c + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

int64_t plan_chunks(int64_t pairs) { return pairs == 0 ? 1 : (pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs); }

// Orders the lanes' LDS accesses within one wave (its LDS instructions run in order; this keeps the compiler's).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// counts[chunk][expert]: kept pairs of each expert in each chunk.
__global__ __launch_bounds__(kPlanThreads) void expert_count_kernel(const int32_t *__restrict__ ids, int64_t pairs,
                                                                    int64_t chunk, int experts,
                                                                    int32_t *__restrict__ counts) {
    extern __shared__ int32_t s_plan[];
    for (int e = threadIdx.x; e < experts; e += blockDim.x) s_plan[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < pairs ? begin + chunk : pairs;
    for (int64_t p = begin + threadIdx.x; p < end; p += blockDim.x) {
        const int e = ids[p];
        if (e >= 0 && e < experts) atomicAdd(&s_plan[e], 1);  // integer: any order gives the same counts
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += blockDim.x)
        counts[static_cast<int64_t>(blockIdx.x) * experts + e] = s_plan[e];
}

// One workgroup a chunk. Each wave owns a contiguous part of the chunk; LDS holds the next row of every (wave, expert)
// and within 64 pairs the lanes of one expert find their order by ballots over the expert's bits.
// single: the only chunk, whose counts the kernel takes from its own waves' counts.
__global__ __launch_bounds__(kPlanThreads) void expert_place_kernel(const int32_t *__restrict__ ids, int64_t pairs,
                                                                    int64_t chunk, int experts, int bits, int single,
                                                                    const int32_t *__restrict__ counts,
                                                                    int32_t *__restrict__ offsets,
                                                                    int32_t *__restrict__ rows,
                                                                    int32_t *__restrict__ row_pairs) {
    extern __shared__ int32_t s_plan[];
    __shared__ int32_t s_wave[kPlanThreads / kWave], s_carry;
    const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    int32_t *next = s_plan + wave * experts;  // [waves][experts]
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < pairs ? begin + chunk : pairs;
    // a wave's part: whole steps of 64, so that the parts stay in order
    const int64_t part = ((end - begin + blockDim.x - 1) / blockDim.x) * kWave;
    const int64_t from = begin + wave * part;
    const int64_t to = from + part < end ? from + part : end;
    int32_t *s_total = s_plan + waves * experts, *s_before = s_total + experts;
    for (int i = threadIdx.x; i < (waves + 2) * experts; i += blockDim.x) s_plan[i] = 0;
    if (threadIdx.x == 0) s_carry = 0;
    __syncthreads();
    for (int64_t p = from + lane; p < to; p += kWave) {
        const int e = ids[p];
        if (e >= 0 && e < experts) atomicAdd(&next[e], 1);
    }
    __syncthreads();
    // every expert's pairs, of all chunks and of those before this one: where there are fewer experts than threads,
    // several threads an expert share the chunks (a read of the counts is a trip to L2, and they are read in turn)
    if (single) {
        for (int e = threadIdx.x; e < experts; e += blockDim.x)
            for (int w = 0; w < waves; ++w) s_total[e] += s_plan[w * experts + e];
    } else {
        const int per = min(1 << bits, static_cast<int>(blockDim.x)), shares = blockDim.x / per;
        for (int e = threadIdx.x % per; e < experts; e += per) {
            int32_t total = 0, before = 0;
#pragma unroll 8
            for (int c = threadIdx.x / per; c < static_cast<int>(gridDim.x); c += shares) {
                const int32_t n = counts[static_cast<int64_t>(c) * experts + e];
                before += c < static_cast<int>(blockIdx.x) ? n : 0;
                total += n;
            }
            atomicAdd(&s_total[e], total);
            atomicAdd(&s_before[e], before);
        }
    }
    __syncthreads();
    // first row of every expert, then of this chunk and of each of its waves
    for (int e0 = 0; e0 < experts; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int32_t total = 0, before = 0;
        if (e < experts) {
            total = s_total[e];
            before = s_before[e];
        }
        const int32_t sum = wave_inclusive_sum(total);
        if (lane == kWave - 1) s_wave[wave] = sum;
        __syncthreads();
        int32_t first = s_carry + sum - total;
        for (int w = 0; w < wave; ++w) first += s_wave[w];
        __syncthreads();
        if (threadIdx.x == blockDim.x - 1) s_carry = first + total;
        if (e < experts) {
            if (blockIdx.x == 0) offsets[e] = first;
            int32_t at = first + before;
            for (int w = 0; w < waves; ++w) {
                const int32_t n = s_plan[w * experts + e];
                s_plan[w * experts + e] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    const int32_t kept = s_carry;
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = kept;
    for (int64_t p0 = from; p0 < to; p0 += kWave) {
        const int64_t p = p0 + lane;
        const int e = p < to ? ids[p] : -1;
        const bool valid = e >= 0 && e < experts;
        uint64_t same = __ballot(valid);
        for (int b = 0; b < bits; ++b) {
            const uint64_t ones = __ballot(valid && ((e >> b) & 1));
            same &= (e >> b) & 1 ? ones : ~ones;
        }
        const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
        int32_t row = -1;
        if (valid) row = next[e] + rank;
        wave_lds_fence();  // every lane has read its counter before one lane moves it on
        if (valid && rank == 0) next[e] = row + __popcll(same);
        wave_lds_fence();
        if (p < to) rows[p] = row;
        if (valid) row_pairs[row] = static_cast<int32_t>(p);
    }
    // the rows past the kept ones that lie in this chunk's range
    for (int64_t r = begin + threadIdx.x; r < end; r += blockDim.x)
        if (r >= kept) row_pairs[r] = -1;
}

// ------------------------------------------------------------------------------------------------------------
// rows

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / kWave;
constexpr int64_t kRowBlocks = 16384;

// Work item i of a walk over tokens: token i / parts, columns [part * 64 V packs, ...) of its row.
struct RowItem {
    int64_t token, col;
};

template <typename T, int V>
__device__ __forceinline__ RowItem row_item(int64_t i, int parts) {
    return {i / parts, (i % parts) * (kWave * V * Pack<T>::kN) + static_cast<int64_t>(threadIdx.x % kWave) * Pack<T>::kN};
}

// ONCE: the row is read or written this one time, and takes no room in the caches from what is read again (a choice by
// measurement: with it in its loads the combine of 32768 x 8 rows of 2048 bf16 takes 205 us instead of 221, and in its
// stores the backward of 30000 x 2 rows of 2000 float32 232 instead of 254; the dispatch's stores and the backward's
// loads are better without. Rows that fit the caches cost it up to 0.7 us a call).
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void load_row(const T *row, int64_t col, int64_t dim, typename Pack<T>::V *v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = col + static_cast<int64_t>(i) * kWave * Pack<T>::kN;
        if (ONCE && c + Pack<T>::kN <= dim)
            v[i] = __builtin_nontemporal_load(reinterpret_cast<const typename Pack<T>::VU *>(row + c));
        else
            v[i] = load_pack(row, c, dim);
    }
}

template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_row(T *row, int64_t col, int64_t dim, const typename Pack<T>::V *v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = col + static_cast<int64_t>(i) * kWave * Pack<T>::kN;
        if (ONCE && c + Pack<T>::kN <= dim)
            __builtin_nontemporal_store(v[i], reinterpret_cast<typename Pack<T>::VU *>(row + c));
        else if (c < dim) store_pack(row, c, dim, v[i]);
    }
}

// Zeros the sorted rows that no pair has; the grid's waves share them.
template <typename T, int V>
__device__ __forceinline__ void zero_tail(T *out, int64_t pairs, int64_t kept, int64_t dim, int parts) {
    typename Pack<T>::V zero[V];
#pragma unroll
    for (int i = 0; i < V; ++i) zero[i] = static_cast<T>(0.0f);
    if (kept < 0) kept = 0;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    for (int64_t i = wave; i < (pairs - kept) * parts; i += static_cast<int64_t>(gridDim.x) * kRowWaves) {
        const RowItem it = row_item<T, V>(i, parts);
        store_row<T, V>(out + (kept + it.token) * dim, it.col, dim, zero);
    }
}

template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void expert_dispatch_kernel(const T *__restrict__ x,
                                                                      const int32_t *__restrict__ kept,
                                                                      const int32_t *__restrict__ rows, int64_t tokens,
                                                                      int64_t choices, int64_t dim, int parts,
                                                                      T *__restrict__ sent) {
    const int64_t pairs = tokens * choices;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    for (int64_t i = wave; i < tokens * parts; i += static_cast<int64_t>(gridDim.x) * kRowWaves) {
        const RowItem it = row_item<T, V>(i, parts);
        typename Pack<T>::V v[V];
        load_row<T, V>(x + it.token * dim, it.col, dim, v);
        for (int64_t k = 0; k < choices; ++k) {
            const int64_t r = rows[it.token * choices + k];
            if (r >= 0 && r < pairs) store_row<T, V>(sent + r * dim, it.col, dim, v);
        }
    }
    zero_tail<T, V>(sent, pairs, *kept, dim, parts);
}

// The rows of a token's kept pairs are read four at a time: each lane first takes one pair's row number and weight, and
// the wave then goes through the kept ones, whose numbers are uniform, so no load waits for another's address.
template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void expert_combine_kernel(const T *__restrict__ source,
                                                                     const int32_t *__restrict__ rows,
                                                                     const float *__restrict__ weights, int64_t tokens,
                                                                     int64_t choices, int64_t dim, int parts,
                                                                     T *__restrict__ y) {
    constexpr int N = Pack<T>::kN, kGroup = 4;
    const int64_t pairs = tokens * choices;
    const int lane = threadIdx.x % kWave;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    for (int64_t i = wave; i < tokens * parts; i += static_cast<int64_t>(gridDim.x) * kRowWaves) {
        const RowItem it = row_item<T, V>(i, parts);
        float acc[V][N] = {};
        for (int64_t k0 = 0; k0 < choices; k0 += kWave) {
            int32_t row = -1;
            float weight = 1.0f;
            if (k0 + lane < choices) {
                row = rows[it.token * choices + k0 + lane];
                if (weights) weight = weights[it.token * choices + k0 + lane];
            }
            uint64_t kept = __ballot(row >= 0 && row < pairs);
            while (kept) {
                typename Pack<T>::V v[kGroup][V];
                float w[kGroup];
                int n = 0;
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    if (kept == 0) break;
                    const int k = __builtin_ctzll(kept);
                    kept &= kept - 1;
                    const int64_t r = __builtin_amdgcn_readlane(row, k);
                    w[q] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), k));
                    load_row<T, V, true>(source + r * dim, it.col, dim, v[q]);
                    n = q + 1;
                }
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    if (q >= n) break;
#pragma unroll
                    for (int a = 0; a < V; ++a)
#pragma unroll
                        for (int j = 0; j < N; ++j)
                            acc[a][j] = __builtin_fmaf(w[q], static_cast<float>(v[q][a][j]), acc[a][j]);
                }
            }
        }
        typename Pack<T>::V o[V];
#pragma unroll
        for (int a = 0; a < V; ++a)
#pragma unroll
            for (int j = 0; j < N; ++j) o[a][j] = static_cast<T>(acc[a][j]);
        store_row<T, V, true>(y + it.token * dim, it.col, dim, o);
    }
}

// One wave a token, all of its columns in turn: the dot products need whole rows. The choices follow each other: the
// token's gradient comes from L1 for all but the first, and with several choices' rows under way at once fewer waves fit
// (16384 x 2 rows of 4096 bf16, with its combine: four at once took a quarter longer, two at once 1%).
template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void expert_combine_bwd_kernel(
    const T *__restrict__ source, const int32_t *__restrict__ kept, const int32_t *__restrict__ rows,
    const float *__restrict__ weights, const T *__restrict__ grad_y, int64_t tokens, int64_t choices, int64_t dim,
    int parts, T *__restrict__ grad_source, float *__restrict__ grad_weights) {
    constexpr int N = Pack<T>::kN;
    const int64_t pairs = tokens * choices;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRowWaves + threadIdx.x / kWave;
    for (int64_t t = wave; t < tokens; t += static_cast<int64_t>(gridDim.x) * kRowWaves) {
        for (int64_t k = 0; k < choices; ++k) {
            const int64_t r = rows[t * choices + k];
            const bool valid = r >= 0 && r < pairs;
            double total = 0.0;  // of the parts' sums: a row may be very long, and a long float32 chain drifts
            float dot = 0.0f;
            if (valid) {
                const float w = weights[t * choices + k];
                for (int part = 0; part < parts; ++part) {
                    const RowItem it = row_item<T, V>(t * parts + part, parts);
                    typename Pack<T>::V g[V], v[V];
                    load_row<T, V>(grad_y + t * dim, it.col, dim, g);
                    load_row<T, V>(source + r * dim, it.col, dim, v);
                    dot = 0.0f;
#pragma unroll
                    for (int a = 0; a < V; ++a)
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const float gf = static_cast<float>(g[a][j]);
                            dot = __builtin_fmaf(gf, static_cast<float>(v[a][j]), dot);
                            v[a][j] = static_cast<T>(w * gf);
                        }
                    store_row<T, V, true>(grad_source + r * dim, it.col, dim, v);
                    total += static_cast<double>(dot);
                }
                dot = group_sum<kWave>(static_cast<float>(total));
            }
            if (threadIdx.x % kWave == 0) grad_weights[t * choices + k] = dot;
        }
    }
    zero_tail<T, V>(grad_source, pairs, *kept, dim, parts);
}

constexpr int64_t kLimit = int64_t(1) << 31;

gs_status check_pairs(const char *name, int64_t tokens, int64_t choices, int experts) {
    if (tokens < 0 || choices < 1 || choices >= kLimit || tokens >= kLimit || tokens * choices >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "%s: need tokens >= 0, choices >= 1 and tokens * choices < 2^31", name);
    if (experts < 1 || experts > kMaxExperts)
        return fail(GS_ERR_INVALID_ARG, "%s: experts = %d outside [1, %d]", name, experts, kMaxExperts);
    return GS_OK;
}

gs_status check_rows(const char *name, int64_t tokens, int64_t choices, int experts, int64_t dim, int dtype) {
    const gs_status bad = check_pairs(name, tokens, choices, experts);
    if (bad != GS_OK) return bad;
    if (dim < 1 || dim >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 1 <= dim < 2^31", name);
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "%s: dtype = %d is no gs_dtype", name, dtype);
    return GS_OK;
}

// Packs a lane holds at once, and the parts of a row that make: as many as the row has, up to four, so that a token's
// whole row is under way at once (32768 x 8 rows of 2048 bf16: the combine with four packs 205 us, with two 211, with
// one 212; the dispatch 236, 228 and 230; combine's backward of 16384 x 2 rows of 4096 bf16 127, 129 and 137).
inline int row_packs(int64_t dim, int pack) {
    const int64_t packs = (dim + pack - 1) / pack;
    return packs <= kWave ? 1 : packs <= 2 * kWave ? 2 : 4;
}
inline int row_parts(int64_t dim, int pack) {
    const int64_t span = static_cast<int64_t>(kWave) * row_packs(dim, pack) * pack;
    return static_cast<int>((dim + span - 1) / span);
}
inline dim3 row_grid(int64_t items) {
    const int64_t blocks = (items + kRowWaves - 1) / kRowWaves;
    return dim3(static_cast<unsigned>(blocks < kRowBlocks ? blocks : kRowBlocks));
}

}  // namespace
}  // namespace gs

using namespace gs;

// Launches kernel<T, V> for the type code and row width; `items`: waves of work for one part count.
#define GS_ROW_LAUNCH_V(kernel, T, V, items, ...)                                                                    \
    hipLaunchKernelGGL((kernel<T, V>), row_grid(items), dim3(kRowThreads), 0, stream, __VA_ARGS__)
#define GS_ROW_LAUNCH(kernel, T, items, ...)                                             \
    do {                                                                                 \
        const int packs_ = row_packs(dim, Pack<T>::kN);                                  \
        if (packs_ == 1) GS_ROW_LAUNCH_V(kernel, T, 1, items, __VA_ARGS__);              \
        else if (packs_ == 2) GS_ROW_LAUNCH_V(kernel, T, 2, items, __VA_ARGS__);         \
        else GS_ROW_LAUNCH_V(kernel, T, 4, items, __VA_ARGS__);                          \
        GS_LAUNCH_TRY(#kernel);                                                          \
        return ok();                                                                     \
    } while (0)

extern "C" size_t gs_expert_plan_workspace_bytes(int64_t tokens, int64_t choices, int experts) {
    if (tokens < 0 || choices < 1 || tokens >= kLimit || choices >= kLimit || tokens * choices >= kLimit ||
        experts < 1 || experts > kMaxExperts)
        return 0;
    const int64_t chunks = plan_chunks(tokens * choices);
    return chunks == 1 ? 0 : static_cast<size_t>(chunks) * static_cast<size_t>(experts) * sizeof(int32_t);
}

extern "C" gs_status gs_expert_plan(const int32_t *ids, int64_t tokens, int64_t choices, int experts,
                                    int32_t *offsets, int32_t *rows, int32_t *pairs, void *workspace,
                                    size_t workspace_bytes, void *stream_handle) {
    const gs_status bad = check_pairs("gs_expert_plan", tokens, choices, experts);
    if (bad != GS_OK) return bad;
    const int64_t n = tokens * choices;
    if (!offsets || (n > 0 && (!ids || !rows || !pairs)))
        return fail(GS_ERR_INVALID_ARG, "gs_expert_plan: a required pointer is NULL");
    const size_t need = gs_expert_plan_workspace_bytes(tokens, choices, experts);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(GS_ERR_WORKSPACE, "gs_expert_plan: need %zu workspace bytes, got %zu", need,
                    workspace ? workspace_bytes : 0);
    const size_t bytes = static_cast<size_t>(n) * sizeof(int32_t);
    const gs_status over = check_apart("gs_expert_plan",
                                       {{"offsets", offsets, (experts + size_t(1)) * sizeof(int32_t)},
                                        {"rows", rows, bytes}, {"pairs", pairs, bytes}, {"workspace", workspace, need}},
                                       {{"ids", ids, bytes}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    const int64_t chunk = plan_chunk(n), chunks = plan_chunks(n);
    const int threads = experts <= kWideExperts ? kPlanThreads : kWideThreads;
    int32_t *counts = static_cast<int32_t *>(workspace);
    const dim3 grid(static_cast<unsigned>(chunks)), block(static_cast<unsigned>(threads));
    if (chunks > 1) {
        hipLaunchKernelGGL(expert_count_kernel, grid, block, static_cast<size_t>(experts) * sizeof(int32_t), stream,
                           ids, n, chunk, experts, counts);
        GS_LAUNCH_TRY("expert_count_kernel");
    }
    const size_t lds = plan_lds(threads, experts);
    if (lds + 1024 > 65536)
        GS_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(expert_place_kernel),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPlanLds)));
    hipLaunchKernelGGL(expert_place_kernel, grid, block, lds, stream, ids, n, chunk, experts, bits_for(experts),
                       chunks == 1 ? 1 : 0, counts, offsets, rows, pairs);
    GS_LAUNCH_TRY("expert_place_kernel");
    return ok();
}

extern "C" gs_status gs_expert_dispatch(const void *x, const int32_t *offsets, const int32_t *rows, int64_t tokens,
                                        int64_t choices, int experts, int64_t dim, int dtype, void *sent,
                                        void *stream_handle) {
    const gs_status bad = check_rows("gs_expert_dispatch", tokens, choices, experts, dim, dtype);
    if (bad != GS_OK) return bad;
    if (tokens == 0) return ok();
    if (!x || !offsets || !rows || !sent)
        return fail(GS_ERR_INVALID_ARG, "gs_expert_dispatch: a required pointer is NULL");
    const size_t row = static_cast<size_t>(dim) * dtype_size(dtype), pairs = static_cast<size_t>(tokens) * choices;
    const gs_status over = check_apart("gs_expert_dispatch", {{"sent", sent, pairs * row}},
                                       {{"x", x, tokens * row},
                                        {"offsets", offsets, (experts + size_t(1)) * sizeof(int32_t)},
                                        {"rows", rows, pairs * sizeof(int32_t)}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    const int32_t *kept = offsets + experts;
    // the copy is of bits, so two instances serve the three types
    if (dtype == GS_F32) {
        const int parts = row_parts(dim, Pack<float>::kN);
        GS_ROW_LAUNCH(expert_dispatch_kernel, float, tokens * parts, static_cast<const float *>(x), kept, rows, tokens,
                      choices, dim, parts, static_cast<float *>(sent));
    }
    const int parts = row_parts(dim, Pack<__bf16>::kN);
    GS_ROW_LAUNCH(expert_dispatch_kernel, __bf16, tokens * parts, static_cast<const __bf16 *>(x), kept, rows, tokens,
                  choices, dim, parts, static_cast<__bf16 *>(sent));
}

extern "C" gs_status gs_expert_combine(const void *source, const int32_t *rows, const float *weights, int64_t tokens,
                                       int64_t choices, int64_t dim, int dtype, void *y, void *stream_handle) {
    const gs_status bad = check_rows("gs_expert_combine", tokens, choices, 1, dim, dtype);
    if (bad != GS_OK) return bad;
    if (tokens == 0) return ok();
    if (!source || !rows || !y) return fail(GS_ERR_INVALID_ARG, "gs_expert_combine: a required pointer is NULL");
    const size_t row = static_cast<size_t>(dim) * dtype_size(dtype), pairs = static_cast<size_t>(tokens) * choices;
    const gs_status over = check_apart("gs_expert_combine", {{"y", y, tokens * row}},
                                       {{"source", source, pairs * row}, {"rows", rows, pairs * sizeof(int32_t)},
                                        {"weights", weights, pairs * sizeof(float)}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
#define GS_COMBINE(T)                                                                                                \
    do {                                                                                                             \
        const int parts = row_parts(dim, Pack<T>::kN);                                                               \
        GS_ROW_LAUNCH(expert_combine_kernel, T, tokens *parts, static_cast<const T *>(source), rows, weights, tokens, \
                      choices, dim, parts, static_cast<T *>(y));                                                     \
    } while (0)
    if (dtype == GS_F32) GS_COMBINE(float);
    if (dtype == GS_BF16) GS_COMBINE(__bf16);
    GS_COMBINE(_Float16);
#undef GS_COMBINE
}

extern "C" gs_status gs_expert_combine_bwd(const void *source, const int32_t *offsets, const int32_t *rows,
                                           const float *weights, const void *grad_y, int64_t tokens, int64_t choices,
                                           int experts, int64_t dim, int dtype, void *grad_source,
                                           float *grad_weights, void *stream_handle) {
    const gs_status bad = check_rows("gs_expert_combine_bwd", tokens, choices, experts, dim, dtype);
    if (bad != GS_OK) return bad;
    if (tokens == 0) return ok();
    if (!source || !offsets || !rows || !weights || !grad_y || !grad_source || !grad_weights)
        return fail(GS_ERR_INVALID_ARG, "gs_expert_combine_bwd: a required pointer is NULL");
    const size_t row = static_cast<size_t>(dim) * dtype_size(dtype), pairs = static_cast<size_t>(tokens) * choices;
    const gs_status over = check_apart("gs_expert_combine_bwd",
                                       {{"grad_source", grad_source, pairs * row},
                                        {"grad_weights", grad_weights, pairs * sizeof(float)}},
                                       {{"source", source, pairs * row},
                                        {"offsets", offsets, (experts + size_t(1)) * sizeof(int32_t)},
                                        {"rows", rows, pairs * sizeof(int32_t)},
                                        {"weights", weights, pairs * sizeof(float)}, {"grad_y", grad_y, tokens * row}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    const int32_t *kept = offsets + experts;
#define GS_COMBINE_BWD(T)                                                                                        \
    do {                                                                                                         \
        const int parts = row_parts(dim, Pack<T>::kN);                                                           \
        GS_ROW_LAUNCH(expert_combine_bwd_kernel, T, tokens, static_cast<const T *>(source), kept, rows, weights, \
                      static_cast<const T *>(grad_y), tokens, choices, dim, parts, static_cast<T *>(grad_source), \
                      grad_weights);                                                                             \
    } while (0)
    if (dtype == GS_F32) GS_COMBINE_BWD(float);
    if (dtype == GS_BF16) GS_COMBINE_BWD(__bf16);
    GS_COMBINE_BWD(_Float16);
#undef GS_COMBINE_BWD
}
