// Layer norm over the last axis and its backward on gfx950.
//
// A group of G lanes holds one row in registers (V packs of 16 bytes a lane), so the mean, the centred sum of squares
// and the output come from one read of the row; the two passes over registers keep the variance exact for rows far
// from zero. The backward forms both row sums from one read of x and grad_y, and every lane keeps the column sums of
// its columns (weight and bias gradient) over all rows that its workgroup visits; the workgroups' sums go to a
// workspace and a second kernel adds them in a fixed order. Wider rows than the registers hold take the kernels that
// read the row again from L2.
//
// Both directions are bound by memory: the forward moves two arrays of x's size and the backward three, and a large
// copy on this card runs at 4.8 TB/s. 32768 x 2048 bf16 forward 48 us (5.5 TB/s), 32768 x 4096 bf16 backward 148 us
// (5.4 TB/s, 7 us of it the second kernel). Below some hundred rows a call is its launches and the host's work.
#include "gs_types.hpp"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 256;           // compute units
constexpr int kWideFwdBlocks = 2048;
constexpr int kWideBwdParts = 64;
constexpr int kBwdBlocks = 768;       // at most: the rows of column sums that the workspace holds
constexpr int kReduceThreads = 1024;
constexpr int kReduceBlocks = 1 << 20;  // at most: a launch has fewer than 2^32 threads

// Floats of a row of column sums in the workspace: whole packs of 16 bytes and cache lines.
__host__ __device__ constexpr int64_t partial_width(int64_t dim) { return (dim + 31) / 32 * 32; }

// Threads of a workgroup whose rows have G lanes each.
constexpr int row_threads(int lanes) { return lanes > kThreads ? lanes : kThreads; }

// Which of the workgroup's rows this thread works on; uniform where a row has whole waves, which keeps row addresses
// out of the lanes' registers.
template <int G>
__device__ __forceinline__ int row_group() {
    const int g = static_cast<int>(threadIdx.x) / G;
    return G >= kWave ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Sum over the G lanes that share a row; slot: LDS words of this sum alone when G spans waves. A row's two sums take
// different slots, so one barrier between writing and reading a slot is enough.
template <int G>
__device__ __forceinline__ float row_sum(float v, float *slot) {
    if constexpr (G <= kWave) {
        return group_sum<G>(v);
    } else {
        v = group_sum<kWave>(v);
        if (threadIdx.x % kWave == 0) slot[threadIdx.x / kWave] = v;
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < G / kWave; ++i) s += slot[i];
        return s;
    }
}

// Two sums at once. Rows that follow each other take two slots in turn: then the one barrier is enough.
template <int G>
__device__ __forceinline__ void row_sums(float &a, float &b, float2 *slot) {
    constexpr int kLanes = G < kWave ? G : kWave;
    a = group_sum<kLanes>(a);
    b = group_sum<kLanes>(b);
    if constexpr (G > kWave) {
        if (threadIdx.x % kWave == 0) slot[threadIdx.x / kWave] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < G / kWave; ++i) {
            a += slot[i].x;
            b += slot[i].y;
        }
    }
}

// Waves of the forward that a SIMD holds at once: 64 registers a wave with up to 8 columns a lane, 80 with 16.
constexpr int fwd_waves(int columns) { return columns > 8 ? 6 : 8; }

template <typename T, typename W, int G, int V>
__global__ __launch_bounds__(row_threads(G), fwd_waves(V * Pack<T>::kN)) void norm_fwd_kernel(
    const T *__restrict__ x, const W *__restrict__ weight, const W *__restrict__ bias, int64_t rows, int dim, float eps,
    T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int N = Pack<T>::kN, kRows = row_threads(G) / G;
    __shared__ float s_sum[2][row_threads(G) / kWave];
    const int lane = threadIdx.x % G;
    const float n = static_cast<float>(dim);
    float w[V * N], b[V * N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (v * G + lane) * N;
        load_floats_long<N>(weight, col, dim, w + v * N);
#pragma unroll
        for (int j = 0; j < N; ++j) b[v * N + j] = 0.0f;
        if (bias) load_floats_long<N>(bias, col, dim, b + v * N);
    }
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + row_group<G>(); r < rows;
         r += static_cast<int64_t>(gridDim.x) * kRows) {
        float c[V * N];
        float s = 0.0f;
        typename Pack<T>::V p[V];
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = read_pack(x + r * dim, (v * G + lane) * N, dim);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = end_pack<T>(p[v], (v * G + lane) * N, dim);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                c[v * N + j] = static_cast<float>(p[v][j]);
                s += c[v * N + j];
            }
        }
        const float m = row_sum<G>(s, s_sum[0]) / n;
        float q = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float &e = c[v * N + j];
                e = (v * G + lane) * N + j < dim ? e - m : 0.0f;
                q = __builtin_fmaf(e, e, q);
            }
        const float rs = 1.0f / sqrtf(row_sum<G>(q, s_sum[1]) / n + eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            typename Pack<T>::V o;
#pragma unroll
            for (int j = 0; j < N; ++j)
                o[j] = static_cast<T>(__builtin_fmaf(c[v * N + j] * rs, w[v * N + j], b[v * N + j]));
            store_pack(y + r * dim, (v * G + lane) * N, dim, o);
        }
        if (mean && lane == 0) {
            mean[r] = m;
            rstd[r] = rs;
        }
    }
}

// Rows wider than the registers hold, or shorter than a pack: one workgroup a row, three reads (the last two from L2). A
// thread adds its packs' sums in float64: a row may be very long, and a long chain of float32 additions of like terms
// drifts (2^24 columns of 0.1: their mean by 6e-4). 4096 x 16384 bf16 76 us either way.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_fwd_wide_kernel(const T *__restrict__ x, const W *__restrict__ weight,
                                                                 const W *__restrict__ bias, int64_t rows, int64_t dim,
                                                                 float eps, T *__restrict__ y,
                                                                 float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int N = Pack<T>::kN;
    __shared__ float s_sum[2][kThreads / kWave];
    const float n = static_cast<float>(dim);
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *row = x + r * dim;
        double s = 0.0;
        for (int64_t col = threadIdx.x * N; col < dim; col += kThreads * N) {
            float c[N], of = 0.0f;
            load_floats<N>(row, col, dim, c);
#pragma unroll
            for (int j = 0; j < N; ++j) of += c[j];
            s += static_cast<double>(of);
        }
        const float m = row_sum<kThreads>(static_cast<float>(s), s_sum[0]) / n;
        double q = 0.0;
        for (int64_t col = threadIdx.x * N; col < dim; col += kThreads * N) {
            float c[N], of = 0.0f;
            load_floats<N>(row, col, dim, c);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float e = col + j < dim ? c[j] - m : 0.0f;
                of = __builtin_fmaf(e, e, of);
            }
            q += static_cast<double>(of);
        }
        const float rs = 1.0f / sqrtf(row_sum<kThreads>(static_cast<float>(q), s_sum[1]) / n + eps);
        for (int64_t col = threadIdx.x * N; col < dim; col += kThreads * N) {
            float c[N], w[N], b[N] = {};
            load_floats<N>(row, col, dim, c);
            load_floats<N>(weight, col, dim, w);
            if (bias) load_floats<N>(bias, col, dim, b);
            typename Pack<T>::V o;
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = static_cast<T>(__builtin_fmaf((c[j] - m) * rs, w[j], b[j]));
            store_pack(y + r * dim, col, dim, o);
        }
        if (mean && threadIdx.x == 0) {
            mean[r] = m;
            rstd[r] = rs;
        }
    }
}

template <typename T, typename W, int G, int V>
__global__ __launch_bounds__(row_threads(G)) void norm_bwd_kernel(const T *__restrict__ x, const W *__restrict__ weight,
                                                            const float *__restrict__ mean,
                                                            const float *__restrict__ rstd,
                                                            const T *__restrict__ grad_y, int64_t rows, int dim,
                                                            T *__restrict__ grad_x, float *__restrict__ partial) {
    constexpr int N = Pack<T>::kN, kRows = row_threads(G) / G;
    __shared__ float2 s_sum[2][row_threads(G) / kWave];
    __shared__ float s_cols[kRows > 1 ? kThreads * (N + 1) : 1];
    const int lane = threadIdx.x % G, group = row_group<G>();
    const float inverse = 1.0f / static_cast<float>(dim);
    float w[V * N], dw[V * N], db[V * N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_floats_long<N>(weight, (v * G + lane) * N, dim, w + v * N);
#pragma unroll
        for (int j = 0; j < N; ++j) dw[v * N + j] = db[v * N + j] = 0.0f;
    }
    int turn = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + group;
    // The next row is on its way while one is worked on: too few rows are in flight on a CU otherwise. Rows pass the
    // caches by (16384 x 4096 float32 129 us, through them 144; the forward, with one array less, is faster through
    // them).
    typename Pack<T>::V px[V], pg[V];
    float pm = 0.0f, pr = 0.0f;
    const auto fetch = [&](int64_t at) {
        pm = mean[at];
        pr = rstd[at];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * G + lane) * N;
            px[v] = read_pack<true>(x + at * dim, col, dim);
            pg[v] = read_pack<true>(grad_y + at * dim, col, dim);
        }
    };
    if (r < rows) fetch(r);
    for (; r < rows; r += step, turn ^= 1) {
        const float m = pm, rs = pr;
        typename Pack<T>::V cx[V], cg[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            cx[v] = end_pack<T>(px[v], (v * G + lane) * N, dim);
            cg[v] = end_pack<T>(pg[v], (v * G + lane) * N, dim);
        }
        if (r + step < rows) fetch(r + step);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // past the row's end 0 itself: (0 - m) * rs may leave float32's range, and times 0 it would be NaN
                const float xh = (v * G + lane) * N + j < dim ? (static_cast<float>(cx[v][j]) - m) * rs : 0.0f;
                const float gy = static_cast<float>(cg[v][j]);
                dw[v * N + j] = __builtin_fmaf(gy, xh, dw[v * N + j]);
                db[v * N + j] += gy;
                const float g = gy * w[v * N + j];  // zero past the row's end, as weight and grad_y are
                s1 += g;
                s2 = __builtin_fmaf(g, xh, s2);
            }
        __builtin_amdgcn_sched_barrier(0);  // nothing but the packed row and the sums is kept over the barrier
        row_sums<G>(s1, s2, s_sum[turn]);
        s1 *= inverse;
        s2 *= inverse;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            // formed anew from the packed row: kept from above, xh and g would take a register each
            u32x4 bx = __builtin_bit_cast(u32x4, cx[v]), bg = __builtin_bit_cast(u32x4, cg[v]);
            asm volatile("" : "+v"(bx), "+v"(bg));
            cx[v] = __builtin_bit_cast(typename Pack<T>::V, bx);
            cg[v] = __builtin_bit_cast(typename Pack<T>::V, bg);
            typename Pack<T>::V o;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float xh = (static_cast<float>(cx[v][j]) - m) * rs;
                const float g = static_cast<float>(cg[v][j]) * w[v * N + j];
                o[j] = static_cast<T>(rs * (g - s1 - xh * s2));
            }
            store_pack(grad_x + r * dim, (v * G + lane) * N, dim, o);
        }
    }
    // the workgroup's column sums: its groups' added in order
    const int64_t width = partial_width(dim);
    float *out = partial + static_cast<int64_t>(blockIdx.x) * 2 * width;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float *acc = (which ? db : dw) + v * N;
            if constexpr (kRows > 1) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < N; ++j) s_cols[threadIdx.x * (N + 1) + j] = acc[j];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        for (int k = 1; k < kRows; ++k) acc[j] += s_cols[(k * G + lane) * (N + 1) + j];
            }
            if (group == 0) {
                const int col = (v * G + lane) * N;
                if (col < width)
#pragma unroll
                    for (int j = 0; j < N; j += 4)
                        *reinterpret_cast<float4 *>(out + which * width + col + j) =
                            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            }
        }
}

// Rows wider than the registers hold, or shorter than a pack: grad_x by one workgroup a row (two reads), and the column
// sums over the rows of one slice (a third). A thread's sums are float64, as the forward's: 4096 x 16384 bf16 189 us, with
// float32 187.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_bwd_wide_kernel(const T *__restrict__ x, const W *__restrict__ weight,
                                                                 const float *__restrict__ mean,
                                                                 const float *__restrict__ rstd,
                                                                 const T *__restrict__ grad_y, int64_t rows,
                                                                 int64_t dim, T *__restrict__ grad_x) {
    constexpr int N = Pack<T>::kN;
    __shared__ float s_sum[2][2][kThreads / kWave];
    const float n = static_cast<float>(dim);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
        const float m = mean[r], rs = rstd[r];
        double t1 = 0.0, t2 = 0.0;
        float s1 = 0.0f, s2 = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t col = threadIdx.x * N; col < dim; col += kThreads * N) {
                float xh[N], g[N], w[N], of1 = 0.0f, of2 = 0.0f;
                load_floats<N>(x + r * dim, col, dim, xh);
                load_floats<N>(grad_y + r * dim, col, dim, g);
                load_floats<N>(weight, col, dim, w);
                typename Pack<T>::V o;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    xh[j] = col + j < dim ? (xh[j] - m) * rs : 0.0f;  // past the end as above
                    g[j] *= w[j];
                    if (pass == 0) {
                        of1 += g[j];
                        of2 = __builtin_fmaf(g[j], xh[j], of2);
                    } else {
                        o[j] = static_cast<T>(rs * (g[j] - s1 - xh[j] * s2));
                    }
                }
                if (pass) store_pack(grad_x + r * dim, col, dim, o);
                t1 += static_cast<double>(of1);
                t2 += static_cast<double>(of2);
            }
            if (pass == 0) {
                s1 = row_sum<kThreads>(static_cast<float>(t1), s_sum[turn][0]) / n;
                s2 = row_sum<kThreads>(static_cast<float>(t2), s_sum[turn][1]) / n;
            }
        }
    }
}

// A workgroup has `cols` columns, kThreads or all of a row that is shorter; its threads left over share the rows of the
// slice, so that the sums of very many narrow rows are no long chains of additions, and are joined through LDS in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_columns_kernel(const T *__restrict__ x, const float *__restrict__ mean,
                                                                const float *__restrict__ rstd,
                                                                const T *__restrict__ grad_y, int64_t rows,
                                                                int64_t dim, int cols, float *__restrict__ partial) {
    __shared__ float2 s_part[kThreads];
    const int shares = kThreads / cols, share = threadIdx.x / cols;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * cols + threadIdx.x % cols;
    const bool mine = share < shares && col < dim;
    double tw = 0.0, tb = 0.0;
    if (mine)
        for (int64_t r = static_cast<int64_t>(blockIdx.y) * shares + share; r < rows;
             r += static_cast<int64_t>(gridDim.y) * shares) {
            const double g = static_cast<double>(static_cast<float>(grad_y[r * dim + col]));
            tw = __builtin_fma(g, static_cast<double>((static_cast<float>(x[r * dim + col]) - mean[r]) * rstd[r]), tw);
            tb += g;
        }
    float dw = static_cast<float>(tw), db = static_cast<float>(tb);
    s_part[threadIdx.x] = make_float2(dw, db);
    __syncthreads();
    if (!mine || share > 0) return;
    for (int i = 1; i < shares; ++i) {
        dw += s_part[i * cols + threadIdx.x].x;
        db += s_part[i * cols + threadIdx.x].y;
    }
    float *out = partial + static_cast<int64_t>(blockIdx.y) * 2 * partial_width(dim);
    out[col] = dw;
    out[partial_width(dim) + col] = db;
}

// grad_weight (y = 0) and grad_bias (y = 1): 64 columns a workgroup, its 16 waves take the partial sums in turn, so
// that many reads are under way over few columns (763 parts of 4096 columns: 25 MB in 7 us, most of them from L2).
template <typename W>
__global__ __launch_bounds__(kReduceThreads) void norm_reduce_kernel(const float *__restrict__ partial, int parts,
                                                                     int64_t dim, W *__restrict__ grad_weight,
                                                                     W *__restrict__ grad_bias) {
    constexpr int kWaves = kReduceThreads / kWave;
    __shared__ float s_part[kWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t width = partial_width(dim);
    for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kWave; c0 < dim; c0 += static_cast<int64_t>(gridDim.x) * kWave) {
        const int64_t col = c0 + lane;
        float s = 0.0f;
        if (col < dim) {
            const float *p = partial + blockIdx.y * width + col;
#pragma unroll 8
            for (int i = wave; i < parts; i += kWaves) s += p[static_cast<int64_t>(i) * 2 * width];
        }
        __syncthreads();  // the columns before are stored
        s_part[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && col < dim) {
            for (int i = 1; i < kWaves; ++i) s += s_part[i][lane];
            (blockIdx.y ? grad_bias : grad_weight)[col] = static_cast<W>(s);
        }
    }
}

// How a row is held: the lanes that share it and the packs of a lane; none: wider than registers hold, or shorter than
// a pack. As few lanes as have two packs or less, so that short rows leave no lane idle and need no barrier. Both sides
// of the borders in bf16, forward and backward: 65536 x 128 with 16 lanes a row 14 and 20 us, with 64 lanes 22 and 38;
// 65536 x 1024 with 64 lanes of two packs 48 and 74 us, with 256 of one 83 and 131; 8192 x 8192 in registers 48 and 79 us,
// by the kernels that read rows again 90 and 188 (16384 x 4096: 48 and 76, 68 and 109).
struct RowShape {
    int lanes, packs;
};

inline RowShape row_shape(int64_t dim, int pack) {
    const int64_t packs = (dim + pack - 1) / pack;
    if (dim < pack) return {0, 0};
    if (packs <= 16) return {16, 1};
    if (packs <= 64) return {64, 1};
    if (packs <= 128) return {64, 2};
    if (packs <= 256) return {256, 1};
    if (packs <= 512) return {256, 2};
    if (packs <= 1024) return {512, 2};
    if (packs <= 2048 && pack == 4) return {1024, 2};
    return {0, 0};
}

// Workgroups that share `need` turns evenly, at most `most` of them.
int64_t even_blocks(int64_t need, int64_t most) {
    const int64_t turns = (need + most - 1) / most;
    return turns == 0 ? 0 : (need + turns - 1) / turns;
}

// Workgroups of the forward: as many as run at once, which visit the rows in turn with their weights in registers.
int64_t fwd_blocks(int64_t rows, int lanes, int columns) {
    const int64_t waves = row_threads(lanes) / kWave, per = row_threads(lanes) / lanes;
    return even_blocks((rows + per - 1) / per, kUnits * 4 * fwd_waves(columns) / waves);
}

// Workgroups of the backward: one a CU at least, for the memory's rate; more, up to what runs at once, only while each
// still has 8 turns, because each writes a row of float32 column sums that the second kernel reads.
int64_t bwd_blocks(int64_t rows, int lanes) {
    const int64_t waves = row_threads(lanes) / kWave, per = row_threads(lanes) / lanes;
    const int64_t need = (rows + per - 1) / per;
    int64_t most = kUnits * (waves < 12 ? 12 / waves : 1);
    if (most > kBwdBlocks) most = kBwdBlocks;
    if (most > need / 8) most = need / 8;
    if (most < kUnits) most = kUnits;
    return even_blocks(need, most);
}

template <typename T, typename W>
gs_status run_fwd(const void *x, const void *weight, const void *bias, int64_t rows, int64_t dim, float eps, void *y,
                  float *mean, float *rstd, hipStream_t stream) {
    const RowShape shape = row_shape(dim, Pack<T>::kN);
#define GS_NORM_FWD(G, V)                                                                                            \
    if (shape.lanes == G && shape.packs == V) {                                                                      \
        hipLaunchKernelGGL((norm_fwd_kernel<T, W, G, V>), dim3(static_cast<unsigned>(                                \
                               fwd_blocks(rows, G, V * Pack<T>::kN))),                                               \
                           dim3(row_threads(G)), 0, stream, static_cast<const T *>(x),                               \
                           static_cast<const W *>(weight), static_cast<const W *>(bias), rows,                       \
                           static_cast<int>(dim), eps, static_cast<T *>(y), mean, rstd);                             \
        GS_LAUNCH_TRY("norm_fwd_kernel");                                                                            \
        return ok();                                                                                                 \
    }
    GS_NORM_FWD(16, 1)
    GS_NORM_FWD(64, 1)
    GS_NORM_FWD(64, 2)
    GS_NORM_FWD(256, 1)
    GS_NORM_FWD(256, 2)
    GS_NORM_FWD(512, 2)
    if constexpr (Pack<T>::kN == 4) {
        GS_NORM_FWD(1024, 2)
    }
#undef GS_NORM_FWD
    hipLaunchKernelGGL((norm_fwd_wide_kernel<T, W>),
                       dim3(static_cast<unsigned>(rows < kWideFwdBlocks ? rows : kWideFwdBlocks)), dim3(kThreads), 0,
                       stream, static_cast<const T *>(x), static_cast<const W *>(weight), static_cast<const W *>(bias), rows,
                       dim, eps, static_cast<T *>(y), mean, rstd);
    GS_LAUNCH_TRY("norm_fwd_wide_kernel");
    return ok();
}

template <typename T, typename W>
gs_status run_bwd(const void *x, const void *weight, const float *mean, const float *rstd, const void *grad_y,
                  int64_t rows, int64_t dim, void *grad_x, void *grad_weight, void *grad_bias, float *partial,
                  hipStream_t stream) {
    const RowShape shape = row_shape(dim, Pack<T>::kN);
    const T *tx = static_cast<const T *>(x), *tg = static_cast<const T *>(grad_y);
    const W *tw = static_cast<const W *>(weight);
    T *to = static_cast<T *>(grad_x);
    // slices of the rows: of short rows as many as the workspace has room for, each of whole turns of a workgroup
    const int cols = static_cast<int>(dim < kThreads ? dim : kThreads);
    const int64_t turns = (rows + kThreads / cols - 1) / (kThreads / cols);
    const int64_t most = dim < kThreads ? kBwdBlocks : kWideBwdParts;
    int64_t parts = turns < most ? turns : most;
#define GS_NORM_BWD(G, V)                                                                                           \
    if (shape.lanes == G && shape.packs == V) {                                                                     \
        parts = bwd_blocks(rows, G);                                                                                \
        if (rows > 0)                                                                                               \
            hipLaunchKernelGGL((norm_bwd_kernel<T, W, G, V>), dim3(static_cast<unsigned>(parts)),                   \
                               dim3(row_threads(G)), 0, stream, tx, tw, mean, rstd, tg, rows, static_cast<int>(dim), \
                               to, partial);                                                                        \
    }
    GS_NORM_BWD(16, 1)
    GS_NORM_BWD(64, 1)
    GS_NORM_BWD(64, 2)
    GS_NORM_BWD(256, 1)
    GS_NORM_BWD(256, 2)
    GS_NORM_BWD(512, 2)
    if constexpr (Pack<T>::kN == 4) {
        GS_NORM_BWD(1024, 2)
    }
#undef GS_NORM_BWD
    GS_LAUNCH_TRY("norm_bwd_kernel");
    if (shape.lanes == 0 && rows > 0) {
        hipLaunchKernelGGL((norm_bwd_wide_kernel<T, W>),
                           dim3(static_cast<unsigned>(rows < kWideFwdBlocks ? rows : kWideFwdBlocks)), dim3(kThreads), 0,
                           stream, tx, tw, mean, rstd, tg, rows, dim, to);
        GS_LAUNCH_TRY("norm_bwd_wide_kernel");
        hipLaunchKernelGGL((norm_columns_kernel<T>),
                           dim3(static_cast<unsigned>((dim + cols - 1) / cols), static_cast<unsigned>(parts)),
                           dim3(kThreads), 0, stream, tx, mean, rstd, tg, rows, dim, cols, partial);
        GS_LAUNCH_TRY("norm_columns_kernel");
    }
    const int64_t blocks = (dim + kWave - 1) / kWave;
    hipLaunchKernelGGL((norm_reduce_kernel<W>),
                       dim3(static_cast<unsigned>(blocks < kReduceBlocks ? blocks : kReduceBlocks),
                            grad_bias ? 2u : 1u),
                       dim3(kReduceThreads), 0, stream, partial, static_cast<int>(parts), dim,
                       static_cast<W *>(grad_weight), static_cast<W *>(grad_bias));
    GS_LAUNCH_TRY("norm_reduce_kernel");
    return ok();
}

constexpr int64_t kLimit = int64_t(1) << 31;

gs_status check_norm(const char *name, int64_t rows, int64_t dim, int dtype, int weight_dtype) {
    if (rows < 0 || rows >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 0 <= rows < 2^31", name);
    if (dim < 1 || dim >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 1 <= dim < 2^31", name);
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "%s: dtype = %d is no gs_dtype", name, dtype);
    if (weight_dtype != dtype && weight_dtype != GS_F32)
        return fail(GS_ERR_INVALID_ARG, "%s: weight_dtype = %d is neither dtype nor GS_F32", name, weight_dtype);
    return GS_OK;
}

}  // namespace
}  // namespace gs

using namespace gs;

// One call of fn<element type, weight type>(...) for the two type codes.
#define GS_NORM_TYPES(fn, ...)                                                                          \
    do {                                                                                                \
        if (dtype == GS_F32) return fn<float, float>(__VA_ARGS__);                                      \
        if (dtype == GS_BF16)                                                                           \
            return weight_dtype == GS_F32 ? fn<__bf16, float>(__VA_ARGS__) : fn<__bf16, __bf16>(__VA_ARGS__); \
        return weight_dtype == GS_F32 ? fn<_Float16, float>(__VA_ARGS__) : fn<_Float16, _Float16>(__VA_ARGS__); \
    } while (0)

extern "C" gs_status gs_layer_norm_fwd(const void *x, const void *weight, const void *bias, int64_t rows, int64_t dim,
                                       float eps, int dtype, int weight_dtype, void *y, float *mean, float *rstd,
                                       void *stream_handle) {
    const gs_status bad = check_norm("gs_layer_norm_fwd", rows, dim, dtype, weight_dtype);
    if (bad != GS_OK) return bad;
    if (!(eps >= 0.0f)) return fail(GS_ERR_INVALID_ARG, "gs_layer_norm_fwd: eps must be >= 0");
    if ((mean == nullptr) != (rstd == nullptr))
        return fail(GS_ERR_INVALID_ARG, "gs_layer_norm_fwd: mean and rstd go together");
    if (rows == 0) return ok();
    if (!x || !weight || !y) return fail(GS_ERR_INVALID_ARG, "gs_layer_norm_fwd: a required pointer is NULL");
    const size_t bytes = static_cast<size_t>(rows) * dim * dtype_size(dtype), wbytes = dim * dtype_size(weight_dtype);
    const gs_status over = check_apart("gs_layer_norm_fwd",
                                       {{"y", y, bytes}, {"mean", mean, rows * sizeof(float)},
                                        {"rstd", rstd, rows * sizeof(float)}},
                                       {{"x", x, bytes}, {"weight", weight, wbytes}, {"bias", bias, wbytes}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    GS_NORM_TYPES(run_fwd, x, weight, bias, rows, dim, eps, y, mean, rstd, stream);
}

extern "C" size_t gs_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    if (rows < 0 || rows >= kLimit || dim < 1 || dim >= kLimit) return 0;
    return static_cast<size_t>(rows < kBwdBlocks ? rows : kBwdBlocks) * 2 *
           static_cast<size_t>(partial_width(dim)) * sizeof(float);
}

extern "C" gs_status gs_layer_norm_bwd(const void *x, const void *weight, const float *mean, const float *rstd,
                                       const void *grad_y, int64_t rows, int64_t dim, int dtype, int weight_dtype,
                                       void *grad_x, void *grad_weight, void *grad_bias, void *workspace,
                                       size_t workspace_bytes, void *stream_handle) {
    const gs_status bad = check_norm("gs_layer_norm_bwd", rows, dim, dtype, weight_dtype);
    if (bad != GS_OK) return bad;
    if (!weight || !grad_weight || (rows > 0 && (!x || !mean || !rstd || !grad_y || !grad_x)))
        return fail(GS_ERR_INVALID_ARG, "gs_layer_norm_bwd: a required pointer is NULL");
    const size_t need = gs_layer_norm_bwd_workspace_bytes(rows, dim);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(GS_ERR_WORKSPACE, "gs_layer_norm_bwd: need %zu workspace bytes, got %zu", need,
                    workspace ? workspace_bytes : 0);
    const size_t bytes = static_cast<size_t>(rows) * dim * dtype_size(dtype), wbytes = dim * dtype_size(weight_dtype);
    const gs_status over =
        check_apart("gs_layer_norm_bwd",
                    {{"grad_x", grad_x, bytes}, {"grad_weight", grad_weight, wbytes}, {"grad_bias", grad_bias, wbytes},
                     {"workspace", workspace, need}},
                    {{"x", x, bytes}, {"weight", weight, wbytes}, {"mean", mean, rows * sizeof(float)},
                     {"rstd", rstd, rows * sizeof(float)}, {"grad_y", grad_y, bytes}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    GS_NORM_TYPES(run_bwd, x, weight, mean, rstd, grad_y, rows, dim, grad_x, grad_weight, grad_bias,
                  static_cast<float *>(workspace), stream);
}
