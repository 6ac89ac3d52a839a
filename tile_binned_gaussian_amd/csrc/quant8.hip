// Values held in 8 bits on gfx950: e4m3 with a power of two for each block of 128 along a row, and back.
//
// A power of two costs no bits (e4m3 rounds relative to the value, whatever the scale) and is what the matrix cores apply
// by themselves. A block's largest magnitude is exact, so is the division by its scale: each value is rounded once.
//
// Bound by memory: 65536 x 4096 bf16 held in 153 us and restored in 129 (5.3 and 6.3 TB/s, part of it from the last-level
// cache); the smallest calls are a launch of 4 us. Transposed 16 x 4096 x 4096 float32 375 us (straight 231): 3.6
// TB/s, read 32 columns of a row at a time.
#include "gs_f8.hpp"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1 << 16;

// A block of 128 columns by L lanes of one pack each.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T *__restrict__ x, int64_t rows, int64_t dim,
                                                            uint8_t *__restrict__ values,
                                                            uint8_t *__restrict__ scales) {
    constexpr int N = Pack<T>::kN, L = kF8Block / N, kPer = kThreads / L;
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const int64_t across = f8_blocks(dim), total = rows * across;
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kPer + group; b < total;
         b += static_cast<int64_t>(gridDim.x) * kPer) {
        const int64_t row = b / across, col = (b - row * across) * kF8Block + lane * N;
        float v[N];
        load_floats<N>(x + row * dim, col, dim, v);
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t f = finite_bits(v[j]);
            most = f > most ? f : most;
        }
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) {
            const uint32_t o = __shfl_xor(most, d, kWave);
            most = o > most ? o : most;
        }
        const int byte = f8_scale(most);
        const float inverse = f8_inverse(byte);
        uint32_t *out = reinterpret_cast<uint32_t *>(values + b * kF8Block + lane * N);
#pragma unroll
        for (int j = 0; j < N; j += 4) out[j / 4] = f8_pack(v[j], v[j + 1], v[j + 2], v[j + 3], inverse);
        if (lane == 0) scales[b] = static_cast<uint8_t>(byte);
    }
}

// Blocks down the columns: x [batch][rows][dim] to values [batch][dim][blocks of rows]. A workgroup takes 128 rows and
// 32 columns through LDS.
constexpr int kTurnCols = 32;
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_turned_kernel(const T *__restrict__ x, int64_t batch, int64_t rows,
                                                                   int64_t dim, uint8_t *__restrict__ values,
                                                                   uint8_t *__restrict__ scales) {
    __shared__ float s_tile[kF8Block][kTurnCols + 1];
    const int64_t down = f8_blocks(rows), across = (dim + kTurnCols - 1) / kTurnCols, total = batch * down * across;
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        const int64_t b = item / (down * across), rest = item - b * down * across, block = rest / across;
        const int64_t row0 = block * kF8Block, col0 = (rest - block * across) * kTurnCols;
        const T *from = x + b * rows * dim;
        __syncthreads();
        for (int i = threadIdx.x; i < kF8Block * kTurnCols; i += kThreads) {
            const int r = i / kTurnCols, c = i % kTurnCols;
            s_tile[r][c] = row0 + r < rows && col0 + c < dim
                               ? static_cast<float>(from[(row0 + r) * dim + col0 + c])
                               : 0.0f;
        }
        __syncthreads();
        // eight lanes a column, sixteen rows each
        const int c = threadIdx.x / 8, part = threadIdx.x % 8;
        uint32_t most = 0;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            v[j] = s_tile[part * 16 + j][c];
            const uint32_t f = finite_bits(v[j]);
            most = f > most ? f : most;
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) {
            const uint32_t o = __shfl_xor(most, d, kWave);
            most = o > most ? o : most;
        }
        if (col0 + c >= dim) continue;
        const int byte = f8_scale(most);
        const float inverse = f8_inverse(byte);
        const int64_t at = (b * dim + col0 + c) * down + block;
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f8_pack(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], inverse);
        *reinterpret_cast<u32x4 *>(values + at * kF8Block + part * 16) = w;
        if (part == 0) scales[at] = static_cast<uint8_t>(byte);
    }
}

// Rounding up to a power of two may leave the type's range: a value that was finite stays so.
template <typename T>
constexpr float kMost = 3.402823466e38f;
template <>
constexpr float kMost<__bf16> = 3.3895313892515355e38f;
template <>
constexpr float kMost<_Float16> = 65504.0f;

template <typename T>
__device__ __forceinline__ T nearest_finite(float v) {
    return static_cast<T>(v > kMost<T> ? kMost<T> : v < -kMost<T> ? -kMost<T> : v);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *__restrict__ values,
                                                              const uint8_t *__restrict__ scales, int64_t rows,
                                                              int64_t dim, T *__restrict__ x) {
    constexpr int N = Pack<T>::kN, L = kF8Block / N, kPer = kThreads / L;
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const int64_t across = f8_blocks(dim), total = rows * across;
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kPer + group; b < total;
         b += static_cast<int64_t>(gridDim.x) * kPer) {
        const int64_t row = b / across, col = (b - row * across) * kF8Block + lane * N;
        const uint32_t *from = reinterpret_cast<const uint32_t *>(values + b * kF8Block + lane * N);
        const float step = f8_step(scales[b]);
        typename Pack<T>::V o;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const int w = static_cast<int>(from[j / 4]);
            o[j] = nearest_finite<T>(__builtin_amdgcn_cvt_f32_fp8(w, 0) * step);
            o[j + 1] = nearest_finite<T>(__builtin_amdgcn_cvt_f32_fp8(w, 1) * step);
            o[j + 2] = nearest_finite<T>(__builtin_amdgcn_cvt_f32_fp8(w, 2) * step);
            o[j + 3] = nearest_finite<T>(__builtin_amdgcn_cvt_f32_fp8(w, 3) * step);
        }
        store_pack(x + row * dim, col, dim, o);
    }
}

constexpr int64_t kLimit = int64_t(1) << 31;

gs_status check_sizes(const char *name, int64_t rows, int64_t dim, int dtype) {
    if (rows < 0 || rows >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 0 <= rows < 2^31", name);
    if (dim < 1 || dim >= kLimit) return fail(GS_ERR_INVALID_ARG, "%s: need 1 <= dim < 2^31", name);
    if (!known_dtype(dtype)) return fail(GS_ERR_INVALID_ARG, "%s: dtype = %d is no gs_dtype", name, dtype);
    return GS_OK;
}

gs_status check_held(const char *name, const void *values) {
    return reinterpret_cast<uintptr_t>(values) % 16
               ? fail(GS_ERR_INVALID_ARG, "%s: values must start at a multiple of 16 bytes", name)
               : GS_OK;
}

inline dim3 block_grid(int64_t blocks, int per) {
    const int64_t want = (blocks + per - 1) / per;
    return dim3(static_cast<unsigned>(want < kMaxBlocks ? want : kMaxBlocks));
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_quantize(const void *x, int64_t batch, int64_t rows, int64_t dim, int transpose, int dtype,
                                    void *values, void *scales, void *stream_handle) {
    const gs_status bad = check_sizes("gs_quantize", rows, dim, dtype);
    if (bad != GS_OK) return bad;
    if (batch < 0 || batch >= kLimit || (batch > 0 && rows >= kLimit / batch + 1) || batch * rows >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "gs_quantize: need batch >= 0 and batch * rows < 2^31");
    if (transpose && batch * dim >= kLimit)
        return fail(GS_ERR_INVALID_ARG, "gs_quantize: need batch * dim < 2^31 to transpose");
    if (batch == 0 || rows == 0) return ok();
    if (!x || !values || !scales) return fail(GS_ERR_INVALID_ARG, "gs_quantize: a required pointer is NULL");
    const gs_status odd = check_held("gs_quantize", values);
    if (odd != GS_OK) return odd;
    const size_t blocks = transpose ? static_cast<size_t>(batch) * dim * f8_blocks(rows)
                                    : static_cast<size_t>(batch) * rows * f8_blocks(dim);
    const size_t bytes = static_cast<size_t>(batch) * rows * dim * dtype_size(dtype);
    const gs_status over = check_apart("gs_quantize", {{"values", values, blocks * kF8Block}, {"scales", scales, blocks}},
                                       {{"x", x, bytes}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    uint8_t *v = static_cast<uint8_t *>(values), *s = static_cast<uint8_t *>(scales);
#define GS_QUANTIZE(T)                                                                                              \
    do {                                                                                                            \
        if (transpose) {                                                                                            \
            const int64_t items = batch * f8_blocks(rows) * ((dim + kTurnCols - 1) / kTurnCols);                    \
            hipLaunchKernelGGL((quantize_turned_kernel<T>), block_grid(items, 1), dim3(kThreads), 0, stream,        \
                               static_cast<const T *>(x), batch, rows, dim, v, s);                                  \
        } else {                                                                                                    \
            hipLaunchKernelGGL((quantize_kernel<T>), block_grid(blocks, kThreads * Pack<T>::kN / kF8Block),         \
                               dim3(kThreads), 0, stream, static_cast<const T *>(x), batch *rows, dim, v, s);       \
        }                                                                                                           \
    } while (0)
    if (dtype == GS_F32) GS_QUANTIZE(float);
    else if (dtype == GS_BF16) GS_QUANTIZE(__bf16);
    else GS_QUANTIZE(_Float16);
#undef GS_QUANTIZE
    GS_LAUNCH_TRY("quantize_kernel");
    return ok();
}

extern "C" gs_status gs_dequantize(const void *values, const void *scales, int64_t rows, int64_t dim, int dtype,
                                      void *x, void *stream_handle) {
    const gs_status bad = check_sizes("gs_dequantize", rows, dim, dtype);
    if (bad != GS_OK) return bad;
    if (rows == 0) return ok();
    if (!x || !values || !scales) return fail(GS_ERR_INVALID_ARG, "gs_dequantize: a required pointer is NULL");
    const gs_status odd = check_held("gs_dequantize", values);
    if (odd != GS_OK) return odd;
    const size_t blocks = static_cast<size_t>(rows) * f8_blocks(dim);
    const gs_status over = check_apart("gs_dequantize",
                                       {{"x", x, static_cast<size_t>(rows) * dim * dtype_size(dtype)}},
                                       {{"values", values, blocks * kF8Block}, {"scales", scales, blocks}});
    if (over != GS_OK) return over;
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    const uint8_t *v = static_cast<const uint8_t *>(values), *s = static_cast<const uint8_t *>(scales);
#define GS_DEQUANTIZE(T)                                                                                          \
    hipLaunchKernelGGL((dequantize_kernel<T>), block_grid(blocks, kThreads * Pack<T>::kN / kF8Block), dim3(kThreads), \
                       0, stream, v, s, rows, dim, static_cast<T *>(x))
    if (dtype == GS_F32) GS_DEQUANTIZE(float);
    else if (dtype == GS_BF16) GS_DEQUANTIZE(__bf16);
    else GS_DEQUANTIZE(_Float16);
#undef GS_DEQUANTIZE
    GS_LAUNCH_TRY("dequantize_kernel");
    return ok();
}
