// Orthogonalised updates on gfx950: Newton-Schulz steps X = a X + (b A + c A A) X, A = X X^T, on matrix cores.
//
// float32 has no matrix-core rate to speak of next to float16's (157 against 2500 TFLOP/s), so every operand is held
// as a pair of float16, high and low part (22 bits together), and a product of two operands is three matrix products,
// high high + high low + low high, summed in float32. The term left out is 2^-22 of the product.
// X holds values scaled by 2^12 and the Gram side by 2^10: entries of X are at most its largest singular value, and
// the scale keeps the low parts of the smallest ones out of float16's subnormals.
#include "gs_types.hpp"

namespace gs {
namespace {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kScaleX = 4096.0f;
constexpr float kScaleA = 1024.0f;
constexpr int kTile = 64;  // output tile of a workgroup; planes are padded to it with zeros
constexpr int kStep = 32;  // columns of both operands staged at a time
constexpr int kThreads = 256;
constexpr int kNormBlocks = 64;

struct Planes {
    _Float16 *hi, *lo;
};

__device__ __forceinline__ void store_pair(const Planes &p, size_t i, float v) {
    const _Float16 h = static_cast<_Float16>(v);
    p.hi[i] = h;
    p.lo[i] = static_cast<_Float16>(v - static_cast<float>(h));
}
__device__ __forceinline__ float load_pair(const Planes &p, size_t i) {
    return static_cast<float>(p.hi[i]) + static_cast<float>(p.lo[i]);
}

// Partial sums of squares of matrix blockIdx.y in float64.
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_norm_kernel(const T *__restrict__ update, int64_t count,
                                                              double *__restrict__ partial) {
    __shared__ double s_part[kThreads];
    const T *u = update + blockIdx.y * count;
    double s = 0.0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const double v = static_cast<double>(static_cast<float>(u[i]));
        s = __builtin_fma(v, v, s);
    }
    s_part[threadIdx.x] = s;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        if (static_cast<int>(threadIdx.x) < d) s_part[threadIdx.x] += s_part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) partial[blockIdx.y * gridDim.x + blockIdx.x] = s_part[0];
}

// X = update / (norm + eps) in both orders: `direct` laid out as the update, `turned` transposed; 64 x 64 tiles,
// zeros in the padding. direct [batch][pm][pn], turned [batch][pn][pm].
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_split_kernel(const T *__restrict__ update,
                                                               const double *__restrict__ partial, int parts, int m,
                                                               int n, int pm, int pn, float eps, Planes direct,
                                                               Planes turned) {
    __shared__ float s_tile[kTile][kTile + 1];
    __shared__ double s_scale;
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < parts; ++i) s += partial[blockIdx.z * parts + i];
        s_scale = static_cast<double>(kScaleX) / (sqrt(s) + static_cast<double>(eps));
    }
    __syncthreads();
    const double scale = s_scale;
    const size_t plane = static_cast<size_t>(pm) * pn;
    const int r0 = blockIdx.y * kTile, c0 = blockIdx.x * kTile;
    const int tc = threadIdx.x % kTile;
    for (int tr = threadIdx.x / kTile; tr < kTile; tr += kThreads / kTile) {
        const int r = r0 + tr, c = c0 + tc;
        float v = 0.0f;
        if (r < m && c < n)
            v = static_cast<float>(
                static_cast<double>(static_cast<float>(update[(static_cast<size_t>(blockIdx.z) * m + r) * n + c])) *
                scale);
        s_tile[tr][tc] = v;
        store_pair(direct, blockIdx.z * plane + static_cast<size_t>(r) * pn + c, v);
    }
    __syncthreads();
    for (int tr = threadIdx.x / kTile; tr < kTile; tr += kThreads / kTile)
        store_pair(turned, blockIdx.z * plane + static_cast<size_t>(c0 + tr) * pm + r0 + tc, s_tile[tc][tr]);
}

enum Product {
    kGram,        // out = P Q^T scaled: A from X
    kPolynomial,  // out = b A + c (P Q^T): the step's matrix from A
    kApply,       // out = a X + P Q^T, and out_t its transpose
};

struct ProductArgs {
    Planes p, q;     // [rows][depth], [cols][depth]
    Planes add;      // [rows][cols]: what the epilogue adds
    Planes out;      // [rows][cols]
    Planes out_t;    // [cols][rows]
    int rows, cols, depth;
    float scale_acc, scale_add;
};

// One 64 x 64 tile of P Q^T a workgroup, a 32 x 32 quarter a wave.
template <int KIND>
__global__ __launch_bounds__(kThreads) void ortho_product_kernel(ProductArgs a) {
    __shared__ _Float16 s_op[2][2][kTile][kStep + 8];  // [P, Q][hi, lo]
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const size_t b = blockIdx.z;
    const size_t p0 = (b * a.rows + blockIdx.y * kTile) * a.depth, q0 = (b * a.cols + blockIdx.x * kTile) * a.depth;
    const int wr = (wave / 2) * 32, wc = (wave % 2) * 32;
    f32x16 acc = {};
    const int sr = threadIdx.x / 4, sc = threadIdx.x % 4 * 8;  // staging: 64 rows of 4 eights
    for (int k0 = 0; k0 < a.depth; k0 += kStep) {
        const size_t off = static_cast<size_t>(sr) * a.depth + k0 + sc;
        const h16x8 v0 = *reinterpret_cast<const h16x8 *>(a.p.hi + p0 + off);
        const h16x8 v1 = *reinterpret_cast<const h16x8 *>(a.p.lo + p0 + off);
        const h16x8 v2 = *reinterpret_cast<const h16x8 *>(a.q.hi + q0 + off);
        const h16x8 v3 = *reinterpret_cast<const h16x8 *>(a.q.lo + q0 + off);
        __syncthreads();
        *reinterpret_cast<h16x8 *>(&s_op[0][0][sr][sc]) = v0;
        *reinterpret_cast<h16x8 *>(&s_op[0][1][sr][sc]) = v1;
        *reinterpret_cast<h16x8 *>(&s_op[1][0][sr][sc]) = v2;
        *reinterpret_cast<h16x8 *>(&s_op[1][1][sr][sc]) = v3;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; k += 16) {
            const int kc = k + lane / 32 * 8;
            const h16x8 ph = *reinterpret_cast<const h16x8 *>(&s_op[0][0][wr + lane % 32][kc]);
            const h16x8 pl = *reinterpret_cast<const h16x8 *>(&s_op[0][1][wr + lane % 32][kc]);
            const h16x8 qh = *reinterpret_cast<const h16x8 *>(&s_op[1][0][wc + lane % 32][kc]);
            const h16x8 ql = *reinterpret_cast<const h16x8 *>(&s_op[1][1][wc + lane % 32][kc]);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl, qh, acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, ql, acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, qh, acc, 0, 0, 0);
        }
    }
    const int col = blockIdx.x * kTile + wc + lane % 32;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int row = blockIdx.y * kTile + wr + i / 4 * 8 + lane / 32 * 4 + i % 4;
        const size_t at = (b * a.rows + row) * a.cols + col;
        float v = acc[i] * a.scale_acc;
        if constexpr (KIND != kGram) v = __builtin_fmaf(a.scale_add, load_pair(a.add, at), v);
        store_pair(a.out, at, v);
        if constexpr (KIND == kApply) store_pair(a.out_t, (b * a.cols + col) * a.rows + row, v);
    }
}

// out [batch][m][n] from the planes that are laid out as it is, [batch][pm][pn].
template <typename T>
__global__ __launch_bounds__(kThreads) void ortho_finish_kernel(Planes x, int m, int n, int pm, int pn,
                                                                T *__restrict__ out) {
    const int64_t count = static_cast<int64_t>(m) * n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / n, c = i % n;
        out[blockIdx.y * count + i] = static_cast<T>(
            load_pair(x, blockIdx.y * static_cast<size_t>(pm) * pn + static_cast<size_t>(r) * pn + c) / kScaleX);
    }
}

inline int64_t padded(int64_t v) { return (v + kTile - 1) / kTile * kTile; }

struct Layout {
    double *partial;
    Planes x, xt[2], gram, poly;
    size_t bytes;
};

Layout lay_out(void *workspace, int64_t batch, int64_t m, int64_t n) {
    const int64_t M = m < n ? m : n, N = m < n ? n : m;
    const size_t xs = static_cast<size_t>(batch) * padded(M) * padded(N);
    const size_t as = static_cast<size_t>(batch) * padded(M) * padded(M);
    Carver c(workspace);
    Layout l;
    l.partial = c.take<double>(static_cast<size_t>(batch) * kNormBlocks);
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

template <typename T>
gs_status run(const void *update, int64_t batch, int64_t m, int64_t n, int steps, float a, float b, float c, float eps,
              void *out, void *workspace, hipStream_t stream) {
    const Layout l = lay_out(workspace, batch, m, n);
    const bool tall = m > n;
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
    hipLaunchKernelGGL((ortho_split_kernel<T>), dim3(pn / kTile, pm / kTile, z), dim3(kThreads), 0, stream, u,
                       l.partial, static_cast<int>(parts), static_cast<int>(m), static_cast<int>(n), pm, pn, eps,
                       tall ? l.xt[at] : l.x, tall ? l.x : l.xt[at]);
    GS_LAUNCH_TRY("ortho_split_kernel");
    for (int s = 0; s < steps; ++s) {
        const dim3 square(M / kTile, M / kTile, z), wide(N / kTile, M / kTile, z);
        ProductArgs g{l.x, l.x, {}, l.gram, {}, M, M, N, kScaleA / (kScaleX * kScaleX), 0.0f};
        hipLaunchKernelGGL((ortho_product_kernel<kGram>), square, dim3(kThreads), 0, stream, g);
        ProductArgs p{l.gram, l.gram, l.gram, l.poly, {}, M, M, M, c / kScaleA, b};
        hipLaunchKernelGGL((ortho_product_kernel<kPolynomial>), square, dim3(kThreads), 0, stream, p);
        ProductArgs y{l.poly, l.xt[at], l.x, l.x, l.xt[1 - at], M, N, M, 1.0f / kScaleA, a};
        hipLaunchKernelGGL((ortho_product_kernel<kApply>), wide, dim3(kThreads), 0, stream, y);
        GS_LAUNCH_TRY("ortho_product_kernel");
        at = 1 - at;
    }
    int64_t blocks = (m * n + kThreads * 4 - 1) / (kThreads * 4);
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL((ortho_finish_kernel<T>), dim3(static_cast<unsigned>(blocks), z), dim3(kThreads), 0, stream,
                       tall ? l.xt[at] : l.x, static_cast<int>(m), static_cast<int>(n), pm, pn,
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
    return lay_out(nullptr, batch, m, n).bytes;
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
    if (!workspace || workspace_bytes < need)
        return fail(GS_ERR_WORKSPACE, "gs_orthogonalize: need %zu workspace bytes, got %zu", need,
                    workspace ? workspace_bytes : 0);
    hipStream_t stream = static_cast<hipStream_t>(stream_handle);
    if (dtype == GS_F32) return run<float>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
    if (dtype == GS_BF16) return run<__bf16>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
    return run<_Float16>(update, batch, m, n, steps, a, b, c, eps, out, workspace, stream);
}
