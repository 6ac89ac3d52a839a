// Orthogonalised updates on gfx950: Newton-Schulz steps X = a X + (b A + c A A) X, A = X X^T, on matrix cores.
//
// float32 has no matrix-core rate to speak of next to float16's (157 against 2500 TFLOP/s), so every operand is held
// as a pair of float16, high and low part (22 bits together), and a product of two operands is three matrix products,
// high high + high low + low high, summed in float32. The term left out is 2^-22 of the product.
// Every step takes both halves, whatever the result's type: with the default coefficients an error of an operand grows
// by up to 122 in twelve steps, and steps on the high halves alone left float16 results up to 50 times their own
// rounding off.
// The time of large matrices is the products' (4096 x 4096: all but 0.05 of 3.5 ms, at 1.2 PFLOP/s, the rate of this
// card's large float16 library product; its matrix cores are busy 0.82 of the time, and its clock falls under the load).
// Small and middling ones are launches and the latency of their chains.
//
// X holds values scaled by 2^12 and the Gram side by 2^8: entries of X are at most its largest singular value and those
// of A its square, so both reach float16's largest value at singular values of 16. The low parts of entries below 2^-15
// of X are float16's subnormals: they are held to 2^-37 itself, not to 22 bits of their own, which is as exact next to
// a norm of 1. A matrix whose norm is far below eps stays small through all steps; its X takes a larger scale
// (x_scale). Its A may then underflow, which counts for nothing next to a.
#include <type_traits>

#include "gs_types.hpp"

namespace gs {
namespace {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kScaleX = 4096.0f;
constexpr float kScaleA = 256.0f;
constexpr int kThreads = 256;
constexpr int kNormBlocks = 512;  // workgroups that share a matrix's norm, at most
constexpr int kPanel = 32;   // rows of a panel; planes are padded to it with zeros both ways
constexpr int kDepth = 16;   // columns of a block
constexpr int kBlock = kPanel * kDepth;  // elements of a block: 1 KB

// A plane holds a matrix [rows][depth] as blocks of 32 rows and 16 columns, [depth / 16][rows / 32][512], each in the
// order in which a wave's lanes hold a matrix-core operand: lane l has row l % 32 and the eight columns from
// l / 32 * 8 on. A block goes from memory to LDS and from LDS to registers as 1 KB in a row: no bank is hit twice,
// whatever the tile. A tile's blocks of the same columns are neighbours in memory, so the workgroups, which go
// through the columns together, spread over all memory channels.
struct Planes {
    _Float16 *hi, *lo;
};

__device__ __forceinline__ size_t block_at(int panel, int block, int rows) {
    return (static_cast<size_t>(block) * (rows / kPanel) + panel) * kBlock;
}

// Element offset of the eight columns from col (a multiple of 8) on of a row.
__device__ __forceinline__ size_t eight_at(int row, int col, int rows) {
    return block_at(row / kPanel, col / kDepth, rows) + (col / 8 % 2 * kPanel + row % kPanel) * 8;
}

template <int N, typename H>
__device__ __forceinline__ void split(const float *v, H &hi, H &lo) {
#pragma unroll
    for (int j = 0; j < N; ++j) hi[j] = static_cast<_Float16>(v[j]);
    // pairs are rounded together and stay packed: seen through, each would be rounded once more by itself
    typedef uint32_t Words __attribute__((ext_vector_type(N / 2)));
    Words w = __builtin_bit_cast(Words, hi);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        uint32_t word = w[j];
        asm volatile("" : "+v"(word));
        w[j] = word;
    }
    hi = __builtin_bit_cast(H, w);
#pragma unroll
    for (int j = 0; j < N; ++j)
        lo[j] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(hi[j]), -1.0f, v[j]));
}

// The scale of a large matrix's X, a power of two: 2^12, or more where a bound of its singular values over all steps
// leaves room below 8 (no bound, NaN among them: 2^12). Up to 2^60, so that its square stays in float32.
__device__ __forceinline__ float x_scale(double norm, double eps, int steps, float a, float b, float c) {
    double s = norm / (norm + eps), most = s;
    for (int k = 0; k < steps && most < 8.0; ++k) {
        s *= fabs(static_cast<double>(a)) +
             s * s * (fabs(static_cast<double>(b)) + s * s * fabs(static_cast<double>(c)));
        if (!(s <= most)) most = s;
    }
    const int room = most < 8.0 ? ilogb(8.0 / most) : 0;
    return ldexpf(kScaleX, room < 48 ? room : 48);
}

// What the products of a matrix take of its scale s.
struct Scales {
    float gram;  // kScaleA / s^2: of the Gram product's sums
    float out;   // 1 / s: of the result
};

// The sum over the workgroup's threads, in every thread.
__device__ __forceinline__ double workgroup_sum(double v, double *s_part) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    if (threadIdx.x % kWave == 0) s_part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) v += s_part[w];
    return v;
}

// Partial sums of squares of matrix blockIdx.y in float64. 4096 x 4096 bf16: 13 us (2.6 TB/s), 0.4% of the call.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_norm_kernel(const T *__restrict__ update, int64_t count,
                                                              double *__restrict__ partial) {
    constexpr int N = Pack<T>::kN;
    __shared__ double s_part[kThreads / kWave];
    const T *u = update + blockIdx.y * count;
    double s = 0.0;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * N; i < count;
         i += static_cast<int64_t>(gridDim.x) * kThreads * N) {
        const typename Pack<T>::V v = load_pack(u, i, count);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const double d = static_cast<double>(static_cast<float>(v[j]));
            s = __builtin_fma(d, d, s);
        }
    }
    s = workgroup_sum(s, s_part);
    if (threadIdx.x == 0) partial[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X = update / (norm + eps) in both orders: `direct` holds the update's rows, `turned` its columns; 64 x 64 elements
// a workgroup, zeros in the padding. Writes the matrix's scales. Bound by memory: 4096 x 4096 bf16 30 us for 168 MB (5.6
// TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_split_kernel(const T *__restrict__ update,
                                                               const double *__restrict__ partial, int parts, int m,
                                                               int n, int pm, int pn, int steps, float a, float b,
                                                               float c, float eps, Planes direct, Planes turned,
                                                               Scales *__restrict__ scales) {
    constexpr int kTile = 64;
    __shared__ float s_tile[kTile][kTile + 1];
    __shared__ double s_part[kThreads / kWave];
    const size_t plane = blockIdx.z * static_cast<size_t>(pm) * pn;
    const int r0 = blockIdx.y * kTile, c0 = blockIdx.x * kTile;
    const int tr = threadIdx.x / kTile, tc = threadIdx.x % kTile;
    constexpr int kTurns = kTile * kTile / kThreads;
    T in[kTurns];  // on their way while the norm is summed
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int r = r0 + tr + i * (kThreads / kTile), c = c0 + tc;
        in[i] = update[(static_cast<size_t>(blockIdx.z) * m + (r < m ? r : m - 1)) * n + (c < n ? c : n - 1)];
    }
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += partial[blockIdx.z * parts + i];
    const double norm = sqrt(workgroup_sum(sum, s_part)), guard = static_cast<double>(eps);
    const float x = x_scale(norm, guard, steps, a, b, c);
    const double scale = static_cast<double>(x) / (norm + guard);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) scales[blockIdx.z] = {kScaleA / (x * x), 1.0f / x};
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int row = tr + i * (kThreads / kTile);
        s_tile[row][tc] = r0 + row < m && c0 + tc < n
                              ? static_cast<float>(static_cast<double>(static_cast<float>(in[i])) * scale)
                              : 0.0f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kTile / 8; i += kThreads) {
        const int row = i % kTile, col = i / kTile * 8;
        float v[8];
        h16x8 hi, lo;
        if (r0 + row < pm && c0 + col < pn) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s_tile[row][col + j];
            split<8>(v, hi, lo);
            const size_t at = plane + eight_at(r0 + row, c0 + col, pm);
            *reinterpret_cast<h16x8 *>(direct.hi + at) = hi;
            *reinterpret_cast<h16x8 *>(direct.lo + at) = lo;
        }
        if (c0 + row < pn && r0 + col < pm) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s_tile[col + j][row];
            split<8>(v, hi, lo);
            const size_t at = plane + eight_at(c0 + row, r0 + col, pn);
            *reinterpret_cast<h16x8 *>(turned.hi + at) = hi;
            *reinterpret_cast<h16x8 *>(turned.lo + at) = lo;
        }
    }
}

// out = scale_acc P Q^T + scale_add add, P [rows][depth], Q [cols][depth]; a Gram product's scale_acc is the matrix's own.
struct ProductArgs {
    Planes p, q;
    Planes add;       // [cols][rows], as `turned`; hi NULL: nothing is added
    Planes straight;  // [rows][cols]
    Planes turned;    // [cols][rows]
    int rows, cols, depth;  // multiples of 32
    int tile_rows, tile_cols;
    int symmetric;    // P = Q and the result is symmetric: tiles of the lower triangle, written to both sides
    const Scales *scales;  // of each matrix
    float scale_acc, scale_add;
    // the last step's: the result itself, [out_rows][out_cols] of out_type for each matrix, in place of planes
    void *out;
    int out_type, out_rows, out_cols;
    int out_turned;   // its rows are the product's columns
    // few tiles of many columns: workgroups that share a tile's sum, and their parts of it [tile][split][64 x 64]
    int splits;
    float *parts;
};

// One block from memory to LDS, 16 bytes a lane, without registers in between. lds: byte address, the same in the
// whole wave; the instruction takes it from m0, which the compiler sets (a write of the statement's own it would not know
// of: m0 is no register that can be named as clobbered). The load counts in vmcnt; only LDS is written, so no register
// waits for it.
__device__ __forceinline__ void load_block(const _Float16 *src, uint32_t lane_bytes, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(lane_bytes), "s"(src) : "memory");
}

// Until at most OUTSTANDING of this wave's loads are under way and its reads of LDS are done, and until every wave of the
// workgroup is here.
template <int OUTSTANDING>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(OUTSTANDING) : "memory");
}

// 4 x 4 transpose of float16 within each quad of lanes: lane q gives its values for rows 0..3 and gets row q's values
// of lanes 0..3.
__device__ __forceinline__ h16x4 quad_transpose(h16x4 v) {
    u32x2 p = __builtin_bit_cast(u32x2, v);
    const int q = threadIdx.x % 4;
    // with the neighbour: lane pairs exchange so that the even one has rows 0 and 2, the odd one rows 1 and 3
    const uint32_t pick = q % 2 ? 0x07060302u : 0x01000504u;
    p.x = __builtin_amdgcn_perm(p.x, __builtin_amdgcn_mov_dpp(p.x, 0xB1, 0xF, 0xF, true), pick);
    p.y = __builtin_amdgcn_perm(p.y, __builtin_amdgcn_mov_dpp(p.y, 0xB1, 0xF, 0xF, true), pick);
    // with the lane two on
    const uint32_t give = q < 2 ? p.y : p.x;
    const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0x4E, 0xF, 0xF, true);
    const u32x2 r = {q < 2 ? p.x : got, q < 2 ? got : p.y};
    return __builtin_bit_cast(h16x4, r);
}

// The same of float32 values.
__device__ __forceinline__ void quad_transpose(float (&v)[4]) {
    const int q = threadIdx.x % 4;
    const auto swap = [](float given, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, given), decltype(ctrl)::value, 0xF, 0xF, true));
    };
#pragma unroll
    for (int k = 0; k < 4; k += 2) {  // with the neighbour: the even lane gets rows 0 and 2, the odd one rows 1 and 3
        const float got = swap(q % 2 ? v[k] : v[k + 1], std::integral_constant<int, 0xB1>());
        v[k + (q % 2 ? 0 : 1)] = got;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // with the lane two on
        const float got = swap(q < 2 ? v[k + 2] : v[k], std::integral_constant<int, 0x4E>());
        if (q < 2) v[k + 2] = got;
        else v[k] = got;
    }
}

// The workgroup's tile: in order on each of the 8 dies, whose L2 then holds the panels that neighbours share.
__device__ __forceinline__ void tile_of(const ProductArgs &a, int &ti, int &tj) {
    const int tiles = gridDim.x, die = blockIdx.x % 8;
    const int t = die * (tiles / 8) + (die < tiles % 8 ? die : tiles % 8) + blockIdx.x / 8;
    // bands of four tile rows, column by column
    if (a.symmetric) {  // of the lower triangle: band k has 8 k k + 2 k tiles before it
        int band = static_cast<int>(sqrtf(static_cast<float>(t) * 0.125f));
        while (8 * band * band + 2 * band > t) --band;
        while (8 * (band + 1) * (band + 1) + 2 * (band + 1) <= t) ++band;
        const int height = a.tile_rows - band * 4 < 4 ? a.tile_rows - band * 4 : 4;
        int in = t - (8 * band * band + 2 * band);
        const int whole = height * (band * 4 + 1);  // in columns that all rows of the band reach
        if (in < whole) {
            ti = in % height;
            tj = in / height;
        } else {
            in -= whole;
            int first = 1;  // the first row of the band that reaches the column
            while (in >= height - first) in -= height - first++;
            ti = first + in;
            tj = band * 4 + first;
        }
        ti += band * 4;
    } else {
        const int band = t / (4 * a.tile_cols), in = t % (4 * a.tile_cols);
        const int height = a.tile_rows - band * 4 < 4 ? a.tile_rows - band * 4 : 4;
        ti = band * 4 + in % height;
        tj = in / height;
    }
}

// What the epilogue adds to four sums of this lane: both halves.
struct Four {
    h16x4 hi, lo;
};

// Where a lane's four sums lie in `turned` and `add`: rows g * 8 + lane / 32 * 4 + 0..3 of row panel mp, column lane % 32
// of column panel np.
__device__ __forceinline__ size_t four_at(const ProductArgs &a, size_t batch, int mp, int np, int g, int lane) {
    return batch * (static_cast<size_t>(a.rows) * a.cols) + block_at(np, mp * 2 + g / 2, a.cols) +
           (g % 2 * kPanel + lane % 32) * 8 + lane / 32 * 4;
}

__device__ __forceinline__ Four load_four(const ProductArgs &a, size_t at) {
    Four f = {};
    if (a.add.hi) {
        f.hi = *reinterpret_cast<const h16x4 *>(a.add.hi + at);
        f.lo = *reinterpret_cast<const h16x4 *>(a.add.lo + at);
    }
    return f;
}

// Four neighbours of a row of the result, those past its end left out.
template <typename T>
__device__ __forceinline__ void store_out(const ProductArgs &a, size_t batch, int row, int col, const float *v) {
    if (row >= a.out_rows || col >= a.out_cols) return;
    T *to = static_cast<T *>(a.out) + (batch * a.out_rows + row) * a.out_cols + col;
    typedef T V __attribute__((ext_vector_type(4)));
    typedef V VU __attribute__((aligned(sizeof(T))));
    if (col + 4 <= a.out_cols) {
        *reinterpret_cast<VU *>(to) = V{static_cast<T>(v[0]), static_cast<T>(v[1]), static_cast<T>(v[2]),
                                        static_cast<T>(v[3])};
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (col + k < a.out_cols) to[k] = static_cast<T>(v[k]);
}

// Four sums on their way out. both: to `turned` too. of: the matrix's scales, read before the first store.
__device__ __forceinline__ void finish_four(const ProductArgs &a, const Scales &of, size_t batch, int mp, int np, int g,
                                            float *v, const Four &add, int lane, bool both) {
    const size_t at = four_at(a, batch, mp, np, g, lane);
    const float scale_acc = a.symmetric && !a.add.hi ? of.gram : a.scale_acc;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v[k] = __builtin_fmaf(a.scale_add, static_cast<float>(add.hi[k]) + static_cast<float>(add.lo[k]),
                              v[k] * scale_acc);
    if (a.out) {
        float r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = v[k] * of.out;
        int row = mp * kPanel + g * 8 + lane / 32 * 4, col = np * kPanel + lane % 32;
        if (a.out_turned) {
            const int down = row;
            row = col;
            col = down;
        } else {
            quad_transpose(r);
            row += lane % 4;
            col = np * kPanel + lane % 32 / 4 * 4;
        }
        if (a.out_type == GS_F32) store_out<float>(a, batch, row, col, r);
        else if (a.out_type == GS_BF16) store_out<__bf16>(a, batch, row, col, r);
        else store_out<_Float16>(a, batch, row, col, r);
        return;
    }
    h16x4 h, l;
    split<4>(v, h, l);
    if (both) {
        *reinterpret_cast<h16x4 *>(a.turned.hi + at) = h;
        *reinterpret_cast<h16x4 *>(a.turned.lo + at) = l;
    }
    // after the transpose this lane: row g * 8 + lane / 32 * 4 + lane % 4, columns from lane % 32 / 4 * 4
    const size_t to = batch * (static_cast<size_t>(a.rows) * a.cols) + block_at(mp, np * 2 + lane % 32 / 16, a.rows) +
                      (lane % 16 / 8 * kPanel + g * 8 + lane / 32 * 4 + lane % 4) * 8 + lane % 8 / 4 * 4;
    *reinterpret_cast<h16x4 *>(a.straight.hi + to) = quad_transpose(h);
    *reinterpret_cast<h16x4 *>(a.straight.lo + to) = quad_transpose(l);
}

// A workgroup of WR x WC waves makes a T x T tile, each wave its part of it. A stage of the LDS ring holds 16 columns of
// both halves; while one is multiplied the next is there already (its operands are read ahead of the barrier) and two
// more are on their way.
// Two or three waves a SIMD, so that one has products to issue where another waits at the barrier: matrix cores busy
// 0.82 of the time with 256 and 192, 0.53 with 180 tiles of 128, where a launch's start and end weigh more. LDS is busy
// 0.21, 0.37 and 0.27 of it, without bank conflicts.
template <int T, int WR, int WC>
__global__ __launch_bounds__(WR *WC *kWave, WR *WC / 4 * (T <= 128 ? 2 : 1)) void ortho_product_kernel(ProductArgs a) {
    constexpr int kStages = 4;
    constexpr int kPanels = T / kPanel;
    constexpr int FR = kPanels / WR, FC = kPanels / WC;  // 32 x 32 results of a wave, each way
    static_assert(FR * WR == kPanels && FC * WC == kPanels, "whole results");
    constexpr int kBlocks = 4 * kPanels;        // of a stage: both halves of the rows' panels and of the columns'
    constexpr int L = kBlocks / (WR * WC);      // blocks a wave loads for a stage
    static_assert(L * WR * WC == kBlocks, "the waves share the loads evenly");
    constexpr uint32_t kStageBytes = kBlocks * kBlock * sizeof(_Float16);
    __shared__ __attribute__((aligned(1024))) _Float16 s_ring[kStages * kBlocks * kBlock];

    int ti, tj;
    tile_of(a, ti, tj);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const size_t batch = blockIdx.y;
    const int row_panels = a.rows / kPanel, col_panels = a.cols / kPanel, blocks = a.depth / kDepth;

    // where this wave's blocks of a stage come from; panels past the edge repeat the last one and are not stored
    const _Float16 *src[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int b = wave * L + i;
        const int panel = b % kPanels, plane = b / kPanels % 2, op = b / (kPanels * 2);
        int at = (op ? tj : ti) * kPanels + panel;
        const int last = (op ? col_panels : row_panels) - 1;
        at = at < last ? at : last;
        const Planes &from = op ? a.q : a.p;
        src[i] = (plane ? from.lo : from.hi) + batch * (static_cast<size_t>(op ? a.cols : a.rows) * a.depth) +
                 block_at(at, 0, op ? a.cols : a.rows);
    }
    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) _Float16 *)s_ring));
    const uint32_t lane_bytes = lane * 16;
    const size_t row_step = static_cast<size_t>(row_panels) * kBlock;
    const size_t col_step = static_cast<size_t>(col_panels) * kBlock;
    int issued = 0;
    const auto issue = [&](int i) {  // block i of this wave's share of stage `issued`
        load_block(src[i], lane_bytes, ring + (issued % kStages) * kStageBytes + (wave * L + i) * 1024);
        // past the end the last stage is loaded again, unused
        if (issued + 1 < blocks) src[i] += wave * L + i < kBlocks / 2 ? row_step : col_step;
    };
    const int wr = wave / WC, wc = wave % WC;
    constexpr int R = 2 * (FR + FC);  // operands of a wave for one block of 16 columns: rows high, low, columns high, low
    h16x8 frag[2][R];
    const auto fetch = [&](const _Float16 *stage_at, int turn, int r) {
        const int op = r < 2 * FR ? 0 : 1, q = r - op * 2 * FR, F = op ? FC : FR, plane = q / F, f = q % F;
        frag[turn][r] = *reinterpret_cast<const h16x8 *>(
            stage_at + ((op * 2 + plane) * kPanels + (op ? wc : wr) * F + f) * kBlock);
    };
    const auto stage_at = [&](int stage) { return s_ring + (stage % kStages) * (kBlocks * kBlock) + lane * 8; };
    f32x16 acc[FR][FC] = {};
    // The products of one block of 16 columns with, in between and in this order, the reads of the next block's
    // operands and the loads of the stage `issued`.
    const auto multiply = [&](int turn, const _Float16 *next) {
        constexpr int M = 3 * FR * FC;
        constexpr int kReads = M > R ? M - M / 4 : M;  // the reads end early enough to be done at the next barrier
#pragma unroll
        for (int x = 0; x < M; ++x) {
#pragma unroll
            for (int r = x * R / kReads; r < (x + 1) * R / kReads && r < R; ++r) fetch(next, 1 - turn, r);
#pragma unroll
            for (int i = x * L / M; i < (x + 1) * L / M; ++i) issue(i);
            const int term = x / (FR * FC), i = x / FC % FR, j = x % FC;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag[turn][(term == 0 ? FR : 0) + i],
                                                               frag[turn][2 * FR + (term == 1 ? FC : 0) + j],
                                                               acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        ++issued;
    };
    for (; issued < kStages - 1; ++issued)
#pragma unroll
        for (int i = 0; i < L; ++i) issue(i);
    wait_and_meet<(kStages - 2) * L>();
#pragma unroll
    for (int r = 0; r < R; ++r) fetch(stage_at(0), 0, r);
    for (int i = 0; i < blocks; i += 2) {
        // two blocks of 16 columns; depth is a multiple of 32. At each meeting the next stage is there and all waves
        // are done with the one before this, whose place the loads then take.
        wait_and_meet<(kStages - 3) * L>();
        multiply(0, stage_at(i + 1));
        wait_and_meet<(kStages - 3) * L>();
        multiply(1, stage_at(i + 2));
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    const bool both = !a.symmetric || ti != tj;  // a tile on the diagonal is its own mirror
    const Scales of = a.scales[batch];
#pragma unroll
    for (int i = 0; i < FR; ++i) {
        const int mp = ti * kPanels + wr * FR + i;
        if (mp >= row_panels) continue;
        // a row of results' additions before its first store: one wait for memory, not one for every four values
        Four add[FC][4];
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const int np = tj * kPanels + wc * FC + j;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                add[j][g] = load_four(a, four_at(a, batch, mp, np < col_panels ? np : col_panels - 1, g, lane));
        }
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const int np = tj * kPanels + wc * FC + j;
            if (np >= col_panels) continue;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = acc[i][j][g * 4 + k];
                finish_four(a, of, batch, mp, np, g, v, add[j][g], lane, both);
            }
        }
    }
}

// Of a 64 x 64 tile: its panel i's group of four rows wave % 4 in its column panel wave / 4, as eight waves finish it.
__device__ __forceinline__ Four load_part_four(const ProductArgs &a, size_t batch, int ti, int tj, int i, int wave,
                                               int lane) {
    const int mp = ti * 2 + i, np = tj * 2 + wave / 4, rows = a.rows / kPanel, cols = a.cols / kPanel;
    return load_four(a, four_at(a, batch, mp < rows ? mp : rows - 1, np < cols ? np : cols - 1, wave % 4, lane));
}
__device__ __forceinline__ void finish_part_four(const ProductArgs &a, const Scales &of, size_t batch, int ti, int tj,
                                                 int i, int wave, int lane, f32x4 sum, const Four &add, bool both) {
    float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    const int mp = ti * 2 + i, np = tj * 2 + wave / 4;
    if (mp < a.rows / kPanel && np < a.cols / kPanel)
        finish_four(a, of, batch, mp, np, wave % 4, v, add, lane, both);
}
__device__ __forceinline__ f32x4 *part_at(const ProductArgs &a, size_t tile, int split, int i, int wave, int lane) {
    return reinterpret_cast<f32x4 *>(a.parts) + ((tile * a.splits + split) * 16 + i * 8 + wave) * kWave + lane;
}

// A 64 x 64 tile by WAVES waves that share its sum: each takes its own range of the columns, for the whole tile, with
// operands straight from memory into registers, whose order a block has (2500 x 1111 f32: 6% of the call less than with
// these tiles through LDS in eight stages; 171 tiles of depth 2528 read 221 MB in 21 us, 10.5 TB/s, 0.74 of it from L2).
// No wave waits for another until the sums are joined through LDS, in order, so the time of a few tiles is not the
// latency of a barrier at every stage. Where there are few tiles, several workgroups share one's columns, because a unit
// draws only so much from L2 (300 x 4000: 15 tiles by 15 units 24 us). Each leaves its part in memory for the kernel
// that joins them. (Joined by the last workgroup to come, a call was slower than without: making the parts visible to it
// costs every unit its L2.)
template <int WAVES, bool SHARED>
__global__ __launch_bounds__(WAVES *kWave) void ortho_product_direct_kernel(ProductArgs a) {
    constexpr int kTile = 64, kPanels = kTile / kPanel;
    __shared__ f32x4 s_sum[WAVES][kPanels * 4][kWave];
    int ti, tj;
    tile_of(a, ti, tj);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const size_t batch = blockIdx.y;
    const int row_panels = a.rows / kPanel, col_panels = a.cols / kPanel, blocks = a.depth / kDepth;
    int first = 0, mine = blocks;  // the workgroup's blocks
    if (SHARED) {
        first = blocks * static_cast<int>(blockIdx.z) / a.splits;
        mine = blocks * static_cast<int>(blockIdx.z + 1) / a.splits - first;
    }
    const int from = first + mine * wave / WAVES, to = first + mine * (wave + 1) / WAVES;
    const _Float16 *src[2][2][kPanels];
#pragma unroll
    for (int op = 0; op < 2; ++op)
#pragma unroll
        for (int plane = 0; plane < 2; ++plane)
#pragma unroll
            for (int f = 0; f < kPanels; ++f) {
                const Planes &p = op ? a.q : a.p;
                const int rows = op ? a.cols : a.rows, last = rows / kPanel - 1;
                const int panel = (op ? tj : ti) * kPanels + f;  // past the edge the last one, not stored
                src[op][plane][f] = (plane ? p.lo : p.hi) + batch * (static_cast<size_t>(rows) * a.depth) +
                                    block_at(panel < last ? panel : last, from, rows) + lane * 8;
            }
    f32x16 acc[kPanels][kPanels] = {};
    // a ring of registers: the loads of kAhead blocks are on their way while one is multiplied
    constexpr int kAhead = 3, kRing = kAhead + 1;
    h16x8 ring[kRing][2][2][kPanels];
    int loaded = from;
    const auto load = [&](int slot) {
#pragma unroll
        for (int op = 0; op < 2; ++op)
#pragma unroll
            for (int plane = 0; plane < 2; ++plane)
#pragma unroll
                for (int f = 0; f < kPanels; ++f) {
                    ring[slot][op][plane][f] = *reinterpret_cast<const h16x8 *>(src[op][plane][f]);
                    // past the end the last block is loaded again, unused
                    if (loaded + 1 < to) src[op][plane][f] += static_cast<size_t>(op ? col_panels : row_panels) * kBlock;
                }
        ++loaded;
    };
    const auto multiply = [&](int slot) {
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int i = 0; i < kPanels; ++i)
#pragma unroll
                for (int j = 0; j < kPanels; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[slot][0][term == 0 ? 1 : 0][i],
                                                                       ring[slot][1][term == 1 ? 1 : 0][j],
                                                                       acc[i][j], 0, 0, 0);
    };
    if (from < to) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load(d);
        int k = from;
        for (; k + kRing <= to; k += kRing) {
#pragma unroll
            for (int d = 0; d < kRing; ++d) {
                load((d + kAhead) % kRing);
                __builtin_amdgcn_sched_barrier(0);
                multiply(d);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
            if (k + d < to) multiply(d);
    }
    const bool both = !a.symmetric || ti != tj;
    const Scales of = a.scales[batch];
    Four add[kPanels];
#pragma unroll
    for (int i = 0; i < kPanels; ++i) add[i] = load_part_four(a, batch, ti, tj, i, wave, lane);
#pragma unroll
    for (int i = 0; i < kPanels; ++i) {
        if (i > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < kPanels; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                s_sum[wave][j * 4 + g][lane] = f32x4{acc[i][j][g * 4], acc[i][j][g * 4 + 1], acc[i][j][g * 4 + 2],
                                                     acc[i][j][g * 4 + 3]};
        __syncthreads();
        static_assert(WAVES == kPanels * 4, "a wave finishes one group of four rows of each panel");
        f32x4 sum = s_sum[0][wave][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += s_sum[w][wave][lane];
        if (SHARED)
            *part_at(a, batch * gridDim.x + blockIdx.x, blockIdx.z, i, wave, lane) = sum;
        else
            finish_part_four(a, of, batch, ti, tj, i, wave, lane, sum, add[i], both);
    }
}

// The sums of a tile that workgroups shared, their parts added in order: half a tile a workgroup.
__global__ __launch_bounds__(8 *kWave) void ortho_join_kernel(ProductArgs a) {
    int ti, tj;
    tile_of(a, ti, tj);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave, i = blockIdx.z;
    const size_t batch = blockIdx.y, tile = batch * gridDim.x + blockIdx.x;
    const Four add = load_part_four(a, batch, ti, tj, i, wave, lane);
    const Scales of = a.scales[batch];
    f32x4 sum = *part_at(a, tile, 0, i, wave, lane);
#pragma unroll 4
    for (int p = 1; p < a.splits; ++p) sum += *part_at(a, tile, p, i, wave, lane);
    finish_part_four(a, of, batch, ti, tj, i, wave, lane, sum, add, !a.symmetric || ti != tj);
}

// out [batch][m][n] from the planes that hold its rows, where there are no steps.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_finish_kernel(Planes x, const Scales *__restrict__ scales, int m,
                                                                int n, int pm, int pn, T *__restrict__ out) {
    // a wave: 8 rows, 64 columns
    const int lane = threadIdx.x % kWave;
    const int row = blockIdx.y * 32 + threadIdx.x / kWave * 8 + lane % 8, col = blockIdx.x * 64 + lane / 8 * 8;
    if (row >= m || col >= n) return;
    const size_t at = blockIdx.z * (static_cast<size_t>(pm) * pn) + eight_at(row, col, pm);
    const h16x8 h = *reinterpret_cast<const h16x8 *>(x.hi + at), l = *reinterpret_cast<const h16x8 *>(x.lo + at);
    T *to = out + (static_cast<size_t>(blockIdx.z) * m + row) * n;
    const float scale = scales[blockIdx.z].out;
    constexpr int N = Pack<T>::kN;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
        typename Pack<T>::V v;
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = static_cast<T>((static_cast<float>(h[i * N + j]) + static_cast<float>(l[i * N + j])) * scale);
        if (col + i * N < n) store_pack(to, col + i * N, n, v);
    }
}

// ------------------------------------------------------------------------------------------------------------
// small matrices: one workgroup a matrix, all steps in one launch
//
// 16 x 96 x 160 f32 30 us, as launches of the kernels above 95; 128 x 128 37 and 99, 32 x 1000 27 and 87. A step is 5.4
// us: six phases with a barrier each. A SIMD's vector instructions take half of it (halves and addresses) and its matrix
// products a third; LDS is busy a third of the time, without bank conflicts (with them, and addresses formed in full: 36
// us).
//
// The 32 x 32 tiles of X are dealt to 16 waves, which keep theirs in float32 registers as the matrix cores leave a
// result (lane: column lane % 32; register 4 g + k: row 8 g + lane / 32 * 4 + k). Once a step every wave puts its
// tiles' halves into LDS, columns as rows: so a lane's four values lie together, the last product reads its operand in
// one piece, and the Gram product, which needs the other order, reads it through LDS's transposing load. A product may
// take its 16 columns in any order as long as both operands take the same: LDS blocks here hold them in the
// registers' order, 0-3, 8-11 (lanes 0-31), 4-7, 12-15 (lanes 32-63).

constexpr int kSmallThreads = 1024;
constexpr int kSmallWaves = kSmallThreads / kWave;
constexpr int kSmallTurns = 2;  // tiles of X a wave holds, at most
constexpr int kSmallLds = 159 * 1024;

// Parts of a Gram tile's sum, so that most waves have one.
constexpr int small_parts(int a) { return a == 1 || a == 2 ? 4 : a == 3 ? 2 : 1; }
constexpr int small_triangle(int a) { return a * (a + 1) / 2; }

// Bytes of LDS: both halves of X [32 a][cols] and of a square matrix [32 a][32 a], and the Gram tiles' parts.
inline int64_t small_lds(int64_t rows, int64_t cols) {
    const int a = static_cast<int>(rows / kPanel);
    return 4 * (rows * cols + rows * rows) + (small_parts(a) - 1) * small_triangle(a) * 4096;
}
inline bool is_small(int64_t rows, int64_t cols) {
    return rows <= 128 && rows / kPanel * (cols / kPanel) <= kSmallTurns * kSmallWaves &&
           small_lds(rows, cols) <= kSmallLds;
}

// Element offset in a block of the small kernel's LDS: half h of its columns, row, and the block's own number k of 16
// columns. Rows are in an order of their own in each half and in odd blocks, so that the transposing load, which reads four
// rows of both halves of two blocks at once, finds them in different banks.
__device__ __forceinline__ int small_at(int h, int row, int k) {
    return (h * kPanel + (row ^ (h * 4) ^ (k % 2 * 8))) * 8;
}

// Where a lane's accesses lie in a block, in elements, formed once for all steps.
struct SmallLane {
    int whole;     // the 16 bytes that a lane stores of a column and reads of an operand, in even blocks
    int straight;  // the 8 bytes of the four rows from 0 on, after the transpose; its block: k
    int across;    // the transposing load's 8 bytes, its block: half
    int k, half;
};
__device__ __forceinline__ SmallLane small_lane(int lane) {
    SmallLane l;
    l.whole = small_at(lane / 32, lane % 32, 0);
    l.k = lane % 32 / 16;
    l.straight = small_at(lane / 4 % 2, lane / 32 * 4 + lane % 4, l.k) + lane / 8 % 2 * 4;
    const int p = lane % 16, chunk = p % 4;
    l.half = lane / 16 % 2;
    l.across = small_at(chunk % 2, lane / 32 * 8 + p / 4, l.half) + chunk / 2 * 4;
    return l;
}

// Stores eight of this lane's values (rows t * 16 + lane / 32 * 4 + 0..3 and the four rows 8 on of row block i, one column
// of column block j) as columns: [columns of the tile][rows of the tile].
__device__ __forceinline__ void small_store_turned(_Float16 *plane, int panels, int i, int j, int t,
                                                   const SmallLane &l, h16x8 v) {
    *reinterpret_cast<h16x8 *>(plane + ((i * 2 + t) * panels + j) * kBlock + (l.whole ^ (t * 64))) = v;
}
// Four of the same values, rows g * 8 + lane / 32 * 4 + 0..3, as [rows of the tile][columns of the tile].
__device__ __forceinline__ void small_store_straight(_Float16 *plane, int panels, int i, int j, int g,
                                                     const SmallLane &l, h16x4 v) {
    *reinterpret_cast<h16x4 *>(plane + ((j * 2 + l.k) * panels + i) * kBlock + (l.straight ^ (g * 64))) =
        quad_transpose(v);
}

// An operand as it lies in LDS: row block `panel` of a plane, its block k of 16 columns.
__device__ __forceinline__ h16x8 small_operand(const _Float16 *plane, int panels, int panel, int k,
                                               const SmallLane &l) {
    return *reinterpret_cast<const h16x8 *>(plane + (k * panels + panel) * kBlock + (l.whole ^ (k % 2 * 64)));
}

// An operand across the order in LDS: the rows are the 32 columns of row block i of X, the columns 16 of its columns
// (half k % 2 of column block k / 2). The transposing load gives each of 16 lanes the values that four of them would
// have read at its place: lane p reads four rows of column p / 4, and gets row p of four columns.
__device__ __forceinline__ h16x8 small_operand_turned(const _Float16 *plane, int k, int across, int across4) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 *LdsPtr;
    const _Float16 *at = plane + k / 2 * kBlock + k % 2 * 128;
    const s16x4 first = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at + across));
    const s16x4 second = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at + across4));
    const h16x4 f = __builtin_bit_cast(h16x4, first), s = __builtin_bit_cast(h16x4, second);
    return __builtin_shufflevector(f, s, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x16 small_multiply(f32x16 acc, h16x8 ph, h16x8 pl, h16x8 qh, h16x8 ql) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl, qh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, ql, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, qh, acc, 0, 0, 0);
}

// One step on the workgroup's matrix: x[t] is tile wave + 16 t, row block tile % A, column block tile / A.
template <int A>
__device__ __forceinline__ void small_step(f32x16 (&x)[kSmallTurns], int col_blocks, float a, float b, float c,
                                           _Float16 *lds, int wave, int lane, const SmallLane &l) {
    constexpr int kTri = small_triangle(A), kParts = small_parts(A);
    _Float16 *xh = lds, *xl = xh + col_blocks * 2 * A * kBlock;
    _Float16 *gh = xl + col_blocks * 2 * A * kBlock, *gl = gh + 2 * A * A * kBlock;
    float *parts = reinterpret_cast<float *>(gl + 2 * A * A * kBlock);
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t) {
        const int tile = wave + t * kSmallWaves;
        if (tile < A * col_blocks)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[8];
                h16x8 hi, lo;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = x[t][u * 8 + k];
                split<8>(v, hi, lo);
                small_store_turned(xh, col_blocks, tile % A, tile / A, u, l, hi);
                small_store_turned(xl, col_blocks, tile % A, tile / A, u, l, lo);
            }
    }
    __syncthreads();
    // wave n: tile n % kTri of the lower triangle, part n / kTri of its sum
    const int tri = wave % kTri, part = wave / kTri;
    const int ti = tri >= 6 ? 3 : tri >= 3 ? 2 : tri >= 1 ? 1 : 0, tj = tri - ti * (ti + 1) / 2;
    f32x16 gram = {};
    if (part < kParts) {
        const int blocks = col_blocks * 2, to = blocks * (part + 1) / kParts;
        const int across = l.across + l.half * col_blocks * kBlock, across4 = across ^ 32;
        const int pi = ti * 2 * col_blocks * kBlock, pj = tj * 2 * col_blocks * kBlock;
#pragma unroll 2
        for (int k = blocks * part / kParts; k < to; ++k) {
            const h16x8 ph = small_operand_turned(xh + pi, k, across, across4);
            const h16x8 qh = small_operand_turned(xh + pj, k, across, across4);
            const h16x8 pl = small_operand_turned(xl + pi, k, across, across4);
            const h16x8 ql = small_operand_turned(xl + pj, k, across, across4);
            gram = small_multiply(gram, ph, pl, qh, ql);
        }
        if (part > 0)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4 *>(parts + (((part - 1) * kTri + tri) * 4 + g) * 256 + lane * 4) =
                    f32x4{gram[g * 4], gram[g * 4 + 1], gram[g * 4 + 2], gram[g * 4 + 3]};
    }
    const auto store = [&](const f32x16 &v16) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float v[8];
            h16x8 hi, lo;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v16[u * 8 + k];
            split<8>(v, hi, lo);
            small_store_turned(gh, A, ti, tj, u, l, hi);
            small_store_turned(gl, A, ti, tj, u, l, lo);
            if (ti != tj)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    small_store_straight(gh, A, ti, tj, u * 2 + g, l,
                                         h16x4{hi[g * 4], hi[g * 4 + 1], hi[g * 4 + 2], hi[g * 4 + 3]});
                    small_store_straight(gl, A, ti, tj, u * 2 + g, l,
                                         h16x4{lo[g * 4], lo[g * 4 + 1], lo[g * 4 + 2], lo[g * 4 + 3]});
                }
        }
    };
    if constexpr (kParts > 1) __syncthreads();
    if (part == 0) {
#pragma unroll
        for (int p = 1; p < kParts; ++p)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(parts + (((p - 1) * kTri + tri) * 4 + g) * 256 +
                                                                 lane * 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) gram[g * 4 + k] += v[k];
            }
#pragma unroll
        for (int e = 0; e < 16; ++e) gram[e] *= kScaleA / (kScaleX * kScaleX);
        store(gram);
    }
    __syncthreads();
    if (part == 0) {
        f32x16 square = {};
#pragma unroll
        for (int k = 0; k < 2 * A; ++k) {
            const h16x8 ph = small_operand(gh, A, ti, k, l), qh = small_operand(gh, A, tj, k, l);
            const h16x8 pl = small_operand(gl, A, ti, k, l), ql = small_operand(gl, A, tj, k, l);
            square = small_multiply(square, ph, pl, qh, ql);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) gram[e] = __builtin_fmaf(b, gram[e], square[e] * (c / kScaleA));
    }
    __syncthreads();  // the step's matrix takes the Gram matrix's place
    if (part == 0) store(gram);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t) {
        const int tile = wave + t * kSmallWaves;
        if (tile < A * col_blocks) {
            f32x16 acc = {};
#pragma unroll
            for (int k = 0; k < 2 * A; ++k) {
                const h16x8 ph = small_operand(gh, A, tile % A, k, l);
                const h16x8 qh = small_operand(xh, col_blocks, tile / A, k, l);
                const h16x8 pl = small_operand(gl, A, tile % A, k, l);
                const h16x8 ql = small_operand(xl, col_blocks, tile / A, k, l);
                acc = small_multiply(acc, ph, pl, qh, ql);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[t][e] = __builtin_fmaf(a, x[t][e], acc[e] * (1.0f / kScaleA));
        }
    }
    __syncthreads();  // the next step's halves take these columns' place
}

// Element access through a buffer descriptor: an offset past the end reads 0 and is not written, so the edges of a
// matrix need no branches.
template <typename T>
struct Buffer {
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ Buffer(const T *base, int count)
        : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(base), 0, count * static_cast<int>(sizeof(T)),
                                                 0x00020000)) {}
    __device__ __forceinline__ float load(int offset) const {
        if constexpr (sizeof(T) == 4)
            return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, offset * 4, 0, 0));
        else
            return static_cast<float>(
                __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(rsrc, offset * 2, 0, 0)));
    }
    __device__ __forceinline__ void store(int offset, float v) const {
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rsrc, offset * 4, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<T>(v)), rsrc, offset * 2,
                                                  0, 0);
    }
};

// rows <= cols: the matrix as the steps see it, transposed from the update where tall.
template <typename T, int A>
__global__ __launch_bounds__(kSmallThreads) void ortho_small_kernel(const T *__restrict__ update, int rows, int cols,
                                                                    int tall, int steps, float a, float b, float c,
                                                                    float eps, T *__restrict__ out) {
    extern __shared__ __attribute__((aligned(16))) _Float16 s_small[];
    __shared__ double s_sum[kSmallWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int col_blocks = (cols + kPanel - 1) / kPanel;
    const size_t base = blockIdx.x * (static_cast<size_t>(rows) * cols);
    const int row_step = tall ? 1 : cols, col_step = tall ? rows : 1;
    // the offset of register e of tile t for lane l: in a wide matrix a row past the last one is past the end by itself
    const auto offset = [=](int l, int t, int e) {
        const int tile = wave + t * kSmallWaves;
        const int row = tile % A * kPanel + l / 32 * 4, col = tile / A * kPanel + l % 32, down = e / 4 * 8 + e % 4;
        const int first = col < cols ? row * row_step + col * col_step : 1 << 28;
        const int at = first + down * row_step;
        return tall && row + down >= rows ? 1 << 28 : at;
    };
    const auto has = [=](int t) { return wave + t * kSmallWaves < A * col_blocks; };  // tile t of this wave
    f32x16 x[kSmallTurns];
    const Buffer<T> from(update + base, rows * cols);
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t) {
        x[t] = f32x16{};
        if (has(t))
#pragma unroll
            for (int e = 0; e < 16; ++e) x[t][e] = from.load(offset(lane, t, e));
    }
    double sum = 0.0;
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t)
        if (has(t))
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const double v = static_cast<double>(x[t][e]);
                sum = __builtin_fma(v, v, sum);
            }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < kSmallWaves; ++w) sum += s_sum[w];
    // the power of two first, which rounds nothing that counts next to the norm: no scale leaves float32's range
    int exponent;
    const float mantissa = static_cast<float>(
        frexp(static_cast<double>(kScaleX) / (sqrt(sum) + static_cast<double>(eps)), &exponent));
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t)
        if (has(t))
#pragma unroll
            for (int e = 0; e < 16; ++e) x[t][e] = ldexpf(x[t][e], exponent) * mantissa;
    SmallLane at = small_lane(lane);
    for (int k = 0; k < steps; ++k) {
        // addresses formed anew from these in every step: kept, they would not fit the registers
        asm volatile("" : "+v"(at.whole), "+v"(at.straight), "+v"(at.across));
        small_step<A>(x, col_blocks, a, b, c, s_small, wave, lane, at);
    }
    const Buffer<T> to(out + base, rows * cols);
    int late = lane;  // offsets formed anew: kept from the loads they would take 32 registers all along
    asm volatile("" : "+v"(late));
#pragma unroll
    for (int t = 0; t < kSmallTurns; ++t)
        if (has(t))
#pragma unroll
            for (int e = 0; e < 16; ++e) to.store(offset(late, t, e), x[t][e] * (1.0f / kScaleX));
}

inline int64_t padded(int64_t v) { return (v + kPanel - 1) / kPanel * kPanel; }

constexpr int kUnits = 256;  // compute units

struct Layout {
    double *partial;
    Scales *scales;
    float *parts;
    Planes x, xt[2], gram, poly;
    size_t bytes;
};

int tile_edge(int64_t batch, int rows, int cols, bool symmetric);

// Workgroups that share the sum of each tile of edge 64: as many as leave no unit without one, with four blocks or more
// for each wave. 300 x 4000 f32: with shared tiles 180 us, without 240; 512 x 4000 207 and 258; 64 x 3000 bf16 103 and
// 142. By two the second launch eats what it gives.
int tile_splits(int64_t tiles, int depth) {
    const int64_t most = kUnits / tiles, work = depth / kDepth / 32;
    const int64_t n = most < work ? most : work;
    return n < 3 ? 1 : n > 16 ? 16 : static_cast<int>(n);
}
int64_t tile_count(int64_t batch, int rows, int cols, int edge, bool symmetric) {
    const int64_t r = (rows + edge - 1) / edge, c = (cols + edge - 1) / edge;
    return batch * (symmetric ? r * (r + 1) / 2 : r * c);
}

Layout lay_out(void *workspace, int64_t batch, int64_t m, int64_t n) {
    const int64_t M = m < n ? m : n, N = m < n ? n : m;
    const size_t xs = static_cast<size_t>(batch) * padded(M) * padded(N);
    const size_t as = static_cast<size_t>(batch) * padded(M) * padded(M);
    Carver c(workspace);
    Layout l;
    l.partial = c.take<double>(static_cast<size_t>(batch) * kNormBlocks);
    l.scales = c.take<Scales>(static_cast<size_t>(batch));
    // the Gram product's parts; the others' sums are as long as it has rows, too short to share where tiles are few
    const int m32 = static_cast<int>(padded(M));
    const int64_t tiles = tile_count(batch, m32, m32, 64, true);
    const int splits = tile_edge(batch, m32, m32, true) == 64 ? tile_splits(tiles, static_cast<int>(padded(N))) : 1;
    l.parts = c.take<float>(splits > 1 ? static_cast<size_t>(tiles) * splits * 64 * 64 : 0);
    const auto planes = [&c](size_t count) {
        Planes p;
        p.hi = c.take<_Float16>(count);
        p.lo = c.take<_Float16>(count);
        return p;
    };
    l.x = planes(xs);
    l.xt[0] = planes(xs);
    l.xt[1] = planes(xs);
    l.gram = planes(as);
    l.poly = planes(as);
    l.bytes = c.used;
    return l;
}

gs_status check_sizes(int64_t batch, int64_t m, int64_t n) {
    if (m < 1 || n < 1 || m > 65536 || n > 65536)
        return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: need 1 <= m, n <= 65536");
    if (batch < 0 || batch > 65535 || batch * m * n >= (int64_t(1) << 40))
        return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: need 0 <= batch <= 65535 and batch * m * n < 2^40");
    return GS_OK;
}

// The tile edge of a product: least rounds of workgroups over the chip, times a tile's entries, times what an entry costs
// in a tile of that edge next to the largest (its operands come through L2 and LDS more often). A round of 252 tiles at
// depth 4096 takes 340 us at 256, 230 at 192, 146 at 128 and 46 at 64: 1.20, 1.71 and 2.18 times the time of an entry.
// The costs are lower, because rounds are seldom full and a tile that has its unit's L2 and clock to itself is faster:
// over 90 shapes for which it matters (130 to 4096 rows and columns, stacks of up to 16) calls took 0.3% longer with
// 1.2, 1.6 and 2.4 and 2.8% longer with 1.2, 1.7 and 2.2 (2% less with 1.18, 1.41 and 3.0).
int tile_edge(int64_t batch, int rows, int cols, bool symmetric) {
    int best = 0;
    double least = 0.0;
    const struct {
        int edge;
        double cost;
    } edges[] = {{256, 1.0}, {192, 1.05}, {128, 1.25}, {64, 2.0}};
    for (const auto &e : edges) {
        const int64_t tiles = tile_count(batch, rows, cols, e.edge, symmetric);
        const double t = static_cast<double>((tiles + kUnits - 1) / kUnits) * e.edge * e.edge * e.cost;
        if (best == 0 || t < least) {
            best = e.edge;
            least = t;
        }
    }
    return best;
}

gs_status product(ProductArgs g, int64_t batch, hipStream_t stream) {
    const int edge = tile_edge(batch, g.rows, g.cols, g.symmetric != 0);
    g.tile_rows = (g.rows + edge - 1) / edge;
    g.tile_cols = (g.cols + edge - 1) / edge;
    const dim3 grid(static_cast<unsigned>(g.symmetric ? g.tile_rows * (g.tile_rows + 1) / 2
                                                      : g.tile_rows * g.tile_cols),
                    static_cast<unsigned>(batch));
#define GS_PRODUCT(T, WR, WC)                                                                                       \
    if (edge == T)                                                                                                 \
    hipLaunchKernelGGL((ortho_product_kernel<T, WR, WC>), grid, dim3(WR * WC * kWave), 0, stream, g)
    if (edge == 64) {
        g.splits = g.symmetric && g.parts
                       ? tile_splits(tile_count(batch, g.rows, g.cols, edge, true), g.depth) : 1;
        const dim3 shared(grid.x, grid.y, static_cast<unsigned>(g.splits));
        if (g.splits > 1) {
            hipLaunchKernelGGL((ortho_product_direct_kernel<8, true>), shared, dim3(8 * kWave), 0, stream, g);
            hipLaunchKernelGGL(ortho_join_kernel, dim3(grid.x, grid.y, 2), dim3(8 * kWave), 0, stream, g);
        } else {
            hipLaunchKernelGGL((ortho_product_direct_kernel<8, false>), shared, dim3(8 * kWave), 0, stream, g);
        }
    }
    GS_PRODUCT(128, 4, 2);
    GS_PRODUCT(192, 6, 2);
    GS_PRODUCT(256, 2, 4);
#undef GS_PRODUCT
    GS_LAUNCH_TRY("ortho_product_kernel");
    return GS_OK;
}

template <typename T>
gs_status run_small(const void *update, int64_t batch, int64_t rows, int64_t cols, bool tall, int steps, float a,
                    float b, float c, float eps, void *out, hipStream_t stream) {
    const int lds = static_cast<int>(small_lds(padded(rows), padded(cols)));
#define GS_SMALL(A)                                                                                                  \
    if (padded(rows) == A * kPanel) {                                                                                \
        if (lds + 1024 > 65536)                                                                                      \
            GS_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(ortho_small_kernel<T, A>),                 \
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds));                  \
        hipLaunchKernelGGL((ortho_small_kernel<T, A>), dim3(static_cast<unsigned>(batch)), dim3(kSmallThreads), lds, \
                           stream, static_cast<const T *>(update), static_cast<int>(rows), static_cast<int>(cols),   \
                           tall ? 1 : 0, steps, a, b, c, eps, static_cast<T *>(out));                                 \
    }
    GS_SMALL(1)
    GS_SMALL(2)
    GS_SMALL(3)
    GS_SMALL(4)
#undef GS_SMALL
    GS_LAUNCH_TRY("ortho_small_kernel");
    return ok();
}

template <typename T>
gs_status run(const void *update, int64_t batch, int64_t m, int64_t n, int steps, float a, float b, float c, float eps,
              void *out, void *workspace, hipStream_t stream) {
    const bool tall = m > n;
    if (is_small(padded(tall ? n : m), padded(tall ? m : n)))
        return run_small<T>(update, batch, tall ? n : m, tall ? m : n, tall, steps, a, b, c, eps, out, stream);
    const Layout l = lay_out(workspace, batch, m, n);
    const int M = static_cast<int>(padded(tall ? n : m)), N = static_cast<int>(padded(tall ? m : n));
    const int pm = static_cast<int>(padded(m)), pn = static_cast<int>(padded(n));
    const unsigned z = static_cast<unsigned>(batch);
    const T *u = static_cast<const T *>(update);
    int64_t parts = (m * n + kThreads * 16 - 1) / (kThreads * 16);
    if (parts > kNormBlocks) parts = kNormBlocks;
    hipLaunchKernelGGL((ortho_norm_kernel<T>), dim3(static_cast<unsigned>(parts), z), dim3(kThreads), 0, stream, u,
                       m * n, l.partial);
    GS_LAUNCH_TRY("ortho_norm_kernel");
    int at = 0;  // which transposed copy is current
    hipLaunchKernelGGL((ortho_split_kernel<T>), dim3((pn + 63) / 64, (pm + 63) / 64, z), dim3(kThreads), 0, stream, u,
                       l.partial, static_cast<int>(parts), static_cast<int>(m), static_cast<int>(n), pm, pn, steps, a, b,
                       c, eps, tall ? l.xt[at] : l.x, tall ? l.x : l.xt[at], l.scales);
    GS_LAUNCH_TRY("ortho_split_kernel");
    for (int s = 0; s < steps; ++s) {
        ProductArgs ops[3] = {
            {l.x, l.x, {}, l.gram, l.gram, M, M, N, 0, 0, 1, l.scales, 0.0f, 0.0f, nullptr, 0, 0, 0, 0, 1, l.parts},
            {l.gram, l.gram, l.gram, l.poly, l.poly, M, M, M, 0, 0, 1, l.scales, c / kScaleA, b, nullptr, 0, 0, 0, 0, 1,
             nullptr},
            {l.poly, l.xt[at], l.xt[at], l.x, l.xt[1 - at], M, N, M, 0, 0, 0, l.scales, 1.0f / kScaleA, a, nullptr, 0, 0,
             0, 0, 1, nullptr}};
        if (s == steps - 1) {
            ops[2].out = out;
            ops[2].out_type = std::is_same<T, float>::value ? GS_F32 : std::is_same<T, __bf16>::value ? GS_BF16 : GS_F16;
            ops[2].out_rows = static_cast<int>(m);
            ops[2].out_cols = static_cast<int>(n);
            ops[2].out_turned = tall ? 1 : 0;
        }
        for (const ProductArgs &op : ops) {
            const gs_status bad = product(op, batch, stream);
            if (bad != GS_OK) return bad;
        }
        at = 1 - at;
    }
    if (steps > 0) return ok();
    hipLaunchKernelGGL((ortho_finish_kernel<T>), dim3((pn + 63) / 64, pm / 32, z), dim3(kThreads), 0, stream,
                       tall ? l.xt[at] : l.x, l.scales, static_cast<int>(m), static_cast<int>(n), pm, pn,
                       static_cast<T *>(out));
    GS_LAUNCH_TRY("ortho_finish_kernel");
    return ok();
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n) {
    if (m < 1 || n < 1 || m > 65536 || n > 65536 || batch < 1 || batch > 65535 || batch * m * n >= (int64_t(1) << 40))
        return 0;
    return is_small(padded(m < n ? m : n), padded(m < n ? n : m)) ? 0 : lay_out(nullptr, batch, m, n).bytes;
}

extern "C" gs_status gs_orthogonalize(const void *update, int64_t batch, int64_t m, int64_t n, int steps, float a,
                                      float b, float c, float eps, int dtype, void *out, void *workspace,
                                      size_t workspace_bytes, void *stream_handle) {
    const gs_status bad = check_sizes(batch, m, n);
    if (bad != GS_OK) return bad;
    if (steps < 0 || steps > 100) return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: need 0 <= steps <= 100");
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: dtype = %d is no gs_dtype", dtype);
    if (!(eps >= 0.0f)) return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: eps must be >= 0");
    if (batch == 0) return ok();
    if (!update || !out) return fail(GS_ERR_INVALID_ARG, "gs_orthogonalize: a required pointer is NULL");
    const size_t need = gs_orthogonalize_workspace_bytes(batch, m, n);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(GS_ERR_WORKSPACE, "gs_orthogonalize: need %zu workspace bytes, got %zu", need,
                    workspace ? workspace_bytes : 0);
    const size_t bytes = static_cast<size_t>(batch) * m * n * dtype_size(dtype);
    const gs_status over = check_apart("gs_orthogonalize", {{"out", out, bytes}, {"workspace", workspace, need}},
                                       {{"update", out == update ? nullptr : update, bytes}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    if (dtype == GS_F32) return run<float>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
    if (dtype == GS_BF16) return run<__bf16>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
    return run<_Float16>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
}
