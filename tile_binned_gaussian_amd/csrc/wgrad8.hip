// Gradient of the experts' weights from activations kept in 8 bits on gfx950:
// out[e][k][n] = sum over the rows r of expert e of x[r, k] grad[r, n].
//
// An e4m3 value times its block's power of two is a bfloat16 without rounding, and float16 and float32 gradients are the
// sums of two and three bfloat16 (11 and 24 bits), so the products run on the bfloat16 matrix cores and lose nothing; they
// are summed in float32. The rows are the sum's own axis: both operands lie in LDS as they come, row by row, and the
// transposing LDS load turns them. Few matrices with many rows each are summed in parts of some rows, which a second
// kernel adds in order.
#include "gs_f8.hpp"

namespace gs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 128;      // columns of x and of grad
constexpr int kDeep = 32;       // rows of a step
constexpr int kThreads = 256;
constexpr int kDies = 8;
constexpr int kUnits = 256;
constexpr int kPlaneBytes = kDeep * kTile * 2;

struct GradArgs {
    const uint8_t *x, *x_scales;
    const void *grad;
    const int32_t *offsets, *pairs;  // NULL: one expert has all rows; sorted row r is row r of x
    int64_t rows, x_rows;
    int choices, experts;
    int dim, cols, blocks;           // k, n, blocks of k
    int64_t chunk;                   // rows of a part; all of them: one part an expert
    int parted;                      // the parts go to the workspace
    float *out;                      // [experts][dim][cols], or the parts [items][dim][cols]
};

__device__ __forceinline__ int64_t within(int64_t v, int64_t low, int64_t high) {
    return v < low ? low : v > high ? high : v;
}

struct Run {
    int expert;
    int64_t begin, end;
};
__device__ __forceinline__ Run run_of(const GradArgs &a, int expert) {
    if (!a.offsets) return {expert, 0, a.rows};
    const int64_t begin = within(a.offsets[expert], 0, a.rows);
    return {expert, begin, within(a.offsets[expert + 1], begin, a.rows)};
}
__device__ __forceinline__ int64_t parts_of(const GradArgs &a, const Run &r) {
    return (r.end - r.begin + a.chunk - 1) / a.chunk;
}

// Part number `item` of all experts' parts; expert = experts: there is none.
__device__ __forceinline__ Run find_part(const GradArgs &a, int64_t item) {
    const int lane = threadIdx.x % kWave;
    int64_t before = 0;
    for (int first = 0; first < a.experts; first += kWave) {
        Run r = {first + lane, 0, 0};
        if (first + lane < a.experts) r = run_of(a, first + lane);
        const int64_t n = parts_of(a, r);
        const int64_t upto = before + wave_inclusive_sum(n);
        const uint64_t past = __ballot(item < upto);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int64_t start = __shfl(r.begin + (item - (upto - n)) * a.chunk, at, kWave);
            const int64_t end = __shfl(r.end, at, kWave);
            return {__builtin_amdgcn_readfirstlane(first + at), start, start + a.chunk < end ? start + a.chunk : end};
        }
        before = __shfl(upto, kWave - 1, kWave);
    }
    return {a.experts, 0, 0};
}

// Bytes from a plane's start to 16 columns (unit of 8) of a row: so placed that the four rows which a transposing load
// takes at once lie in different banks.
__device__ __forceinline__ int unit_at(int row, int unit) { return row * (kTile * 2) + (unit ^ (row % 4 * 2)) * 32; }

__device__ __forceinline__ float leading8(float v) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u);
}

// 16 of a row's values as P planes of bfloat16 whose sum they are: each takes the 8 leading bits of what is left, cut off
// and not rounded, so that the largest numbers stay finite. An infinity or NaN is the first plane alone.
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 2;
template <>
constexpr int kPlanes<__bf16> = 1;

template <int P>
__device__ __forceinline__ void split16(const float *v, bf16x8 (&out)[P][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float rest = v[h * 8 + j];
            if constexpr (P > 1) {
                const bool number = finite_bits(rest) != 0 || rest == 0.0f;
                out[0][h][j] = static_cast<__bf16>(number ? leading8(rest) : rest);
                rest = number ? rest - leading8(rest) : 0.0f;
#pragma unroll
                for (int p = 1; p < P; ++p) {
                    out[p][h][j] = static_cast<__bf16>(leading8(rest));
                    rest -= leading8(rest);
                }
            } else {
                out[0][h][j] = static_cast<__bf16>(rest);
            }
        }
}

// One tile of one part: 4 waves of 64 x 64 results.
template <typename T>
__global__ __launch_bounds__(kThreads, 2) void weight_grad_kernel(GradArgs a, int64_t items) {
    constexpr int P = kPlanes<T>, kBytes = (1 + P) * kPlaneBytes;
    __shared__ __attribute__((aligned(1024))) uint8_t s_planes[2 * kBytes];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int wr = wave / 2, wc = wave % 2;
    const int64_t down = f8_blocks(a.dim), across = (a.cols + kTile - 1) / kTile;
    const int64_t tiles = items * down * across;
    const int my_row = threadIdx.x / 8, my_unit = threadIdx.x % 8;
    const int my_place = unit_at(my_row, my_unit);
    // a transposing load: lane p of 16 reads 4 of the 16 columns of row p / 4
    const int p = lane % 16, from = unit_at(lane / 32 * 8 + p / 4, lane / 16 % 2) + p % 4 * 8;

    for (int64_t turn = 0; turn < tiles; turn += gridDim.x) {
        const int64_t now = tiles - turn < gridDim.x ? tiles - turn : gridDim.x;
        const int64_t share = (now + kDies - 1) / kDies;
        const int64_t j = blockIdx.x / kDies, place = blockIdx.x % kDies * share + j;
        if (j >= share || place >= now) return;
        const int64_t tile = turn + place, item = tile / (down * across), rest = tile - item * down * across;
        const int d0 = static_cast<int>(rest / across) * kTile, n0 = static_cast<int>(rest % across) * kTile;
        Run run;
        if (a.parted) run = find_part(a, item);
        else run = run_of(a, static_cast<int>(item));
        if (run.expert >= a.experts) return;  // fewer parts than there could be
        f32x16 acc[2][2] = {};

        u32x4 x_now = {};
        float step = 0.0f, g_now[16];
        const auto load = [&](int64_t first) {
            const int64_t r = first + my_row;
            x_now = u32x4{0, 0, 0, 0};
            step = 1.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) g_now[k] = 0.0f;
            if (r < run.end) {
                int64_t s = r;
                if (a.pairs) s = within(a.pairs[r] / a.choices, 0, a.x_rows - 1);
                x_now = *reinterpret_cast<const u32x4 *>(a.x + (s * a.blocks + d0 / kTile) * kF8Block + my_unit * 16);
                step = f8_step(a.x_scales[s * a.blocks + d0 / kTile]);
                load_floats<16>(static_cast<const T *>(a.grad) + r * a.cols, n0 + my_unit * 16, a.cols, g_now);
            }
        };
        const auto keep = [&](uint8_t *planes) {
            bf16x8 v[2];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int w = static_cast<int>(x_now[k / 4]);
                const float f = k % 4 == 0   ? __builtin_amdgcn_cvt_f32_fp8(w, 0)
                                : k % 4 == 1 ? __builtin_amdgcn_cvt_f32_fp8(w, 1)
                                : k % 4 == 2 ? __builtin_amdgcn_cvt_f32_fp8(w, 2)
                                             : __builtin_amdgcn_cvt_f32_fp8(w, 3);
                v[k / 8][k % 8] = static_cast<__bf16>(f * step);
            }
            *reinterpret_cast<bf16x8 *>(planes + my_place) = v[0];
            *reinterpret_cast<bf16x8 *>(planes + my_place + 16) = v[1];
            bf16x8 g[P][2];
            split16<P>(g_now, g);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                *reinterpret_cast<bf16x8 *>(planes + (1 + q) * kPlaneBytes + my_place) = g[q][0];
                *reinterpret_cast<bf16x8 *>(planes + (1 + q) * kPlaneBytes + my_place + 16) = g[q][1];
            }
        };
        const auto operand = [&](const uint8_t *plane, int unit, int deep) {
            typedef __attribute__((address_space(3))) s16x4 *LdsPtr;
            // the unit's number is even: its place is that of unit 0 or 1, moved
            const uint8_t *at = plane + deep * (kTile * 2) + (from ^ (unit * 32));
            const s16x4 low = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at));
            const s16x4 high = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at + 4 * (kTile * 2)));
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            const s16x8 both = __builtin_shufflevector(low, high, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, both);
        };

        __syncthreads();
        load(run.begin);
        int at = 0;
        for (int64_t first = run.begin; first < run.end; first += kDeep, at ^= 1) {
            uint8_t *planes = s_planes + at * kBytes;
            keep(planes);
            __syncthreads();
            load(first + kDeep);  // zeros past the end
#pragma unroll
            for (int deep = 0; deep < kDeep; deep += 16) {
                bf16x8 d[2], n[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) d[i] = operand(planes, wr * 4 + i * 2, deep);
#pragma unroll
                for (int q = P - 1; q >= 0; --q) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) n[i] = operand(planes + (1 + q) * kPlaneBytes, wc * 4 + i * 2, deep);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            acc[i][k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d[i], n[k], acc[i][k], 0, 0, 0);
                }
            }
        }
        float *out = a.out + (a.parted ? item : run.expert) * static_cast<int64_t>(a.dim) * a.cols;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int n = n0 + wc * 64 + k * 32 + lane % 32;
#pragma unroll
                for (int g = 0; g < 16; ++g) {
                    const int d = d0 + wr * 64 + i * 32 + g / 4 * 8 + lane / 32 * 4 + g % 4;
                    if (d < a.dim && n < a.cols) out[static_cast<int64_t>(d) * a.cols + n] = acc[i][k][g];
                }
            }
    }
}

// Adds each expert's parts in order.
__global__ __launch_bounds__(kThreads) void weight_grad_join_kernel(GradArgs a, const float *__restrict__ parts,
                                                                    int64_t items, int64_t groups, float *__restrict__ out) {
    const int lane = threadIdx.x % kWave;
    const int64_t size = static_cast<int64_t>(a.dim) * a.cols;
    for (int64_t item = blockIdx.x; item < groups * a.experts; item += gridDim.x) {
        const int expert = static_cast<int>(item / groups);
        int64_t first = 0;
        for (int e = lane; e < expert; e += kWave) first += parts_of(a, run_of(a, e));
#pragma unroll
        for (int d = kWave / 2; d > 0; d >>= 1) first += __shfl_xor(first, d, kWave);
        int64_t count = parts_of(a, run_of(a, expert));
        if (first + count > items) count = items - first;  // offsets that are no plan's: what there is room for
        const int64_t i = (item - expert * groups) * kThreads + threadIdx.x;
        if (i >= size) continue;
        const float *from = parts + first * size + i;
        float s = 0.0f;
        for (int64_t k = 0; k < count; ++k) s += from[k * size];
        out[expert * size + i] = s;
    }
}

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int kMaxExperts = 4096;

// Rows of a part and the parts that there can be; one part an expert where its tiles alone fill the chip.
struct Parts {
    int64_t chunk, items;
    bool parted;
};
Parts parts_for(int64_t rows, int experts, int64_t dim, int64_t cols) {
    const int64_t tiles = f8_blocks(dim) * ((cols + kTile - 1) / kTile);
    const int64_t want = 4 * kUnits / tiles;  // parts in all, for four tiles a compute unit
    int64_t chunk = want > 0 ? (rows + want - 1) / want : rows;
    chunk = (chunk + kDeep - 1) / kDeep * kDeep;
    chunk = chunk < 8 * kDeep ? 8 * kDeep : chunk;
    if (experts * tiles >= 2 * kUnits || chunk >= rows) return {rows > 0 ? rows : 1, experts, false};
    return {chunk, rows / chunk + experts, true};
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_expert_weight_grad_workspace_bytes(int64_t rows, int experts, int64_t dim, int64_t cols) {
    if (rows < 0 || rows >= kLimit || experts < 1 || experts > kMaxExperts || dim < 1 || dim >= kLimit || cols < 1 ||
        cols >= kLimit)
        return 0;
    const Parts p = parts_for(rows, experts, dim, cols);
    return p.parted ? static_cast<size_t>(p.items) * dim * cols * sizeof(float) : 0;
}

extern "C" gs_status gs_expert_weight_grad(const void *x, const void *x_scales, const void *grad,
                                              const int32_t *offsets, const int32_t *pairs, int64_t rows,
                                              int64_t x_rows, int64_t choices, int experts, int64_t dim, int64_t cols,
                                              int dtype, float *out, void *workspace, size_t workspace_bytes,
                                              void *stream_handle) {
    const char *name = "gs_expert_weight_grad";
    if (rows < 0 || rows >= kLimit || x_rows < 0 || x_rows >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "%s: need 0 <= rows, x_rows < 2^31", name);
    if (experts < 1 || experts > kMaxExperts)
        return fail(GS_ERR_INVALID_ARG, "%s: experts = %d outside [1, %d]", name, experts, kMaxExperts);
    if (!offsets && experts != 1) return fail(GS_ERR_INVALID_ARG, "%s: offsets may be NULL for one expert only", name);
    if (dim < 1 || dim >= kLimit || cols < 1 || cols >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "%s: need 1 <= dim, cols < 2^31", name);
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "%s: dtype = %d is no gs_dtype", name, dtype);
    if (choices < 1 || choices >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 1 <= choices < 2^31", name);
    if (pairs ? x_rows * choices != rows : x_rows != rows)
        return fail(GS_ERR_INVALID_ARG, "%s: x_rows = %lld do not go with rows = %lld", name,
                    static_cast<long long>(x_rows), static_cast<long long>(rows));
    if (!out || (rows > 0 && (!x || !x_scales || !grad)))
        return fail(GS_ERR_INVALID_ARG, "%s: a required pointer is NULL", name);
    if (reinterpret_cast<uintptr_t>(x) % 16)
        return fail(GS_ERR_INVALID_ARG, "%s: values must start at a multiple of 16 bytes", name);
    const Parts parts = parts_for(rows, experts, dim, cols);
    const size_t size = static_cast<size_t>(dim) * cols * sizeof(float);
    const size_t need = parts.parted ? parts.items * size : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(GS_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", name, need,
                    workspace ? workspace_bytes : 0);
    const size_t blocks = static_cast<size_t>(f8_blocks(dim));
    const gs_status over = check_apart(
        name, {{"out", out, experts * size}, {"workspace", workspace, need}},
        {{"x", x, x_rows * blocks * kF8Block}, {"x_scales", x_scales, x_rows * blocks},
         {"grad", grad, static_cast<size_t>(rows) * cols * dtype_size(dtype)},
         {"offsets", offsets, (experts + size_t(1)) * 4}, {"pairs", pairs, static_cast<size_t>(rows) * 4}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    GradArgs a = {static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(x_scales), grad, offsets, pairs, rows,
                  x_rows, static_cast<int>(choices), experts, static_cast<int>(dim), static_cast<int>(cols),
                  static_cast<int>(blocks), parts.chunk, parts.parted ? 1 : 0,
                  parts.parted ? static_cast<float *>(workspace) : out};
    const int64_t tiles = parts.items * f8_blocks(dim) * ((cols + kTile - 1) / kTile);
    const int64_t whole = (tiles + kDies - 1) / kDies * kDies, most = 1 << 20;
    const dim3 grid(static_cast<unsigned>(whole < most ? whole : most));
    if (dtype == GS_F32)
        hipLaunchKernelGGL((weight_grad_kernel<float>), grid, dim3(kThreads), 0, stream, a, parts.items);
    else if (dtype == GS_BF16)
        hipLaunchKernelGGL((weight_grad_kernel<__bf16>), grid, dim3(kThreads), 0, stream, a, parts.items);
    else
        hipLaunchKernelGGL((weight_grad_kernel<_Float16>), grid, dim3(kThreads), 0, stream, a, parts.items);
    GS_LAUNCH_TRY("weight_grad_kernel");
    if (parts.parted) {
        const int64_t groups = (dim * cols + kThreads - 1) / kThreads, joins = groups * experts;
        hipLaunchKernelGGL(weight_grad_join_kernel, dim3(static_cast<unsigned>(joins < most ? joins : most)),
                           dim3(kThreads), 0, stream, a, static_cast<const float *>(workspace), parts.items, groups, out);
        GS_LAUNCH_TRY("weight_grad_join_kernel");
    }
    return ok();
}
