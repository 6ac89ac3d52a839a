// Gradient of the experts' weights from activations kept in 8 bits on gfx950:
// out[e][k][n] = sum over the rows r of expert e of x[r, k] grad[r, n].
//
// An e4m3 value times its block's power of two is a bfloat16 without rounding (a multiple of 2^-133 up to its largest is),
// and float16 and float32 gradients are the sums of two and three bfloat16 (11 bits, and 24 down to 2^-133), so the products
// run on the bfloat16 matrix cores and lose nothing; they are summed in float32. The rows are the sum's own axis: both
// operands lie in LDS as they come, row by row, and the transposing LDS load turns them. Few matrices with many rows each
// are summed in parts of some rows, which a second kernel adds in order.
//
// 16384 tokens, 2 choices of 16 experts, 4096 x 4096: bf16 1175 to 1236 us, 1.1 to 1.2 PFLOP/s inside a tile (a bfloat16
// library product of one such matrix 1.38), and 18 us a tile for its start and its 256 KB of results, during which its unit
// has no other (both from the times of two numbers of rows); the 91 to 120 registers that a lane of these tiles spills are
// written and read there. 16 x 2048 rows float16 3150 us, float32 3590, 4080 for 4095 columns. 200000 tokens, 2 of 8,
// 128 x 256 bf16: 50 us at 4.5 TB/s and 8.5 for the parts' join.
#include <utility>

#include "gs_f8.hpp"

namespace gs {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kBand = 8;        // tiles of x's columns that are worked on together
constexpr int kSmall = 128, kLarge = 256;  // columns of a tile, of x and of grad
constexpr int kDeep = 32;       // rows of a step
constexpr int kSegment = 1024;  // rows whose places in x are looked up at once
constexpr int kThreads = 256;
constexpr int kDies = 8;
constexpr int kUnits = 256;

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

// Bytes from a plane's start to 8 columns (a chunk) of a row of TILE: so placed that the four rows which a transposing load
// takes at once lie in different banks, and the even or odd chunks of two neighbouring rows too, which are written at once.
template <int TILE>
__device__ __forceinline__ int chunk_at(int row, int chunk) {
    return row * (TILE * 2) + (chunk ^ (row % 4 * 4) ^ (row % 2)) * 16;
}

__device__ __forceinline__ float leading8(float v) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u);
}

// 16 of a row's values as P planes of bfloat16 whose sum they are: each takes the 8 leading bits of what is left, cut off
// and not rounded, so that the largest numbers stay finite. An infinity or NaN is the first plane alone.
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 2;
template <>
constexpr int kPlanes<__bf16> = 1;

// 8 values as P planes.
template <int P, typename V>
__device__ __forceinline__ void split8(const V *packs, bf16x8 (&out)[P]) {
    constexpr int N = sizeof(V) / sizeof((*packs)[0]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (P == 1) {
            out[0][j] = packs[j / N][j % N];
        } else {
            float rest = static_cast<float>(packs[j / N][j % N]);
            const bool number = finite_bits(rest) != 0 || rest == 0.0f;
            out[0][j] = static_cast<__bf16>(number ? leading8(rest) : rest);
            rest = number ? rest - leading8(rest) : 0.0f;
#pragma unroll
            for (int p = 1; p < P; ++p) {
                out[p][j] = static_cast<__bf16>(leading8(rest));
                rest -= leading8(rest);
            }
        }
    }
}

// f(0) to f(N - 1), each with its number as a constant: the compiler's own unrolling gives up on a step as long as that of
// a large tile of float32 rows that end inside a pack, and what it does not unroll keeps its accumulators in memory
// (16 x 2048 rows 4096 x 4095: 132 ms, so 4.1).
template <int... I, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, const F &f) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(const F &f) {
    unrolled(std::make_integer_sequence<int, N>(), f);
}

// One tile of one part: 4 waves of 32 F x 32 F results. A step's rows go as bfloat16 to LDS kAhead steps ahead, and from
// memory to registers one step before that. CUT: rows of grad end inside a pack. NARROW: they are shorter than one.
template <typename T, int F, bool CUT, bool NARROW>
__global__ __launch_bounds__(kThreads, F == 2 ? 2 : 1) void weight_grad_kernel(GradArgs a, int64_t items) {
    constexpr int P = kPlanes<T>, kTile = 64 * F, kRuns = F / 2;  // columns of a tile; a thread's runs of 16 of a row
    constexpr int kPlaneBytes = kDeep * kTile * 2, kBytes = (1 + P) * kPlaneBytes;
    // steps whose rows are in LDS beside the current one's: two where there is room, so that no step begins with a wait
    constexpr int kAhead = 3 * kBytes + kSegment * 8 <= 159 * 1024 / (F == 2 ? 2 : 1) ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) uint8_t s_planes[(kAhead + 1) * kBytes];
    __shared__ int64_t s_rows[kSegment];  // first blocks of the rows of x
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    const int wr = wave / 2, wc = wave % 2;
    const int64_t down = (int64_t{a.dim} + kTile - 1) / kTile, across = (int64_t{a.cols} + kTile - 1) / kTile;
    const int64_t each = down * across, tiles = items * each;
    const int my_row = threadIdx.x / 8, my_col = threadIdx.x % 8 * 16;  // and 128 on
    const int my_place = chunk_at<kTile>(my_row, threadIdx.x % 8 * 2);
    // a transposing load: lane p of 16 reads 4 of the 16 columns of row p / 4
    const int p = lane % 16, from = chunk_at<kTile>(lane / 32 * 8 + p / 4, lane / 16 % 2 * 2 + p / 2 % 2) + p % 2 * 8;

    for (int64_t turn = 0; turn < tiles; turn += gridDim.x) {
        // of each 256 tiles, which run at about the same time, every die takes neighbouring ones: its L2 holds their rows
        const int64_t group = turn + blockIdx.x / kUnits * kUnits;
        const int64_t now = tiles - group < kUnits ? tiles - group : kUnits, share = (now + kDies - 1) / kDies;
        const int64_t j = blockIdx.x % kUnits / kDies, place = blockIdx.x % kDies * share + j;
        if (j >= share || place >= now) return;
        const int64_t tile = group + place, item = tile / each, of = tile - item * each;
        const int64_t band = of / (kBand * across), rest = of - band * kBand * across;
        const int64_t height = down - band * kBand < kBand ? down - band * kBand : kBand;
        const int d0 = static_cast<int>(band * kBand + rest % height) * kTile;
        const int n0 = static_cast<int>(rest / height) * kTile;
        Run run;
        if (a.parted) run = find_part(a, item);
        else run = run_of(a, static_cast<int>(item));
        if (run.expert >= a.experts) return;  // fewer parts than there could be
        f32x16 acc[F][F] = {};

        // Rows and columns past the ends are read at the last one: no load waits for a branch. The rows become zeros on
        // their way to LDS, the columns belong to results that are not stored.
        constexpr int kPacks = 16 / Pack<T>::kN;
        u32x4 x[2][kRuns];
        int step[2][kRuns];
        typename Pack<T>::V g[2][kRuns][kPacks];
        bf16x8 d[2][F], n[2][F];
        for (int64_t start = run.begin; start < run.end; start += kSegment) {
            const int64_t end = start + kSegment < run.end ? start + kSegment : run.end;
            const int count = static_cast<int>(end - start);
            __syncthreads();  // the last rows' operands and places are read
            for (int i = threadIdx.x; i < count; i += kThreads) {
                const int64_t r = start + i;
                s_rows[i] = (a.pairs ? within(a.pairs[r] / a.choices, 0, a.x_rows - 1) : r) * a.blocks;
            }
            __syncthreads();
            // where the step that is loaded next has this thread's row, and the last row there is
            const T *row = static_cast<const T *>(a.grad) + (start + (my_row < count ? my_row : count - 1)) * a.cols;
            const T *const last_row = static_cast<const T *>(a.grad) + (end - 1) * a.cols;
            const int64_t row_step = static_cast<int64_t>(kDeep) * a.cols;
            int64_t source = s_rows[my_row < count ? my_row : count - 1];
            const auto load = [&](int at, int j) {
                const int64_t b = source + (d0 / kF8Block + j < a.blocks ? d0 / kF8Block + j : a.blocks - 1);
                step[at][j] = a.x_scales[b];
                x[at][j] = *reinterpret_cast<const u32x4 *>(a.x + b * kF8Block + my_col);
#pragma unroll
                for (int k = 0; k < kPacks; ++k) {
                    const int col = n0 + j * 128 + my_col + k * Pack<T>::kN;
                    if constexpr (NARROW) {
#pragma unroll
                        for (int q = 0; q < Pack<T>::kN; ++q)
                            g[at][j][k][q] = row[col + q < a.cols ? col + q : a.cols - 1];
                    } else {
                        g[at][j][k] = read_pack(row, col, a.cols);
                    }
                }
            };
            const auto seek = [&](int next) {  // the step from row `next` on is loaded next
                row = row + row_step < last_row ? row + row_step : last_row;
                const int i = next + my_row;
                source = s_rows[i < count ? i : count - 1];
            };
            const auto load_all = [&](int next, int at) {
#pragma unroll
                for (int j = 0; j < kRuns; ++j) load(at, j);
                seek(next);
            };
            // Piece 0, 2, ...: 8 columns of x; 1, 3, ...: of grad. A row past the end is the last one again, with zeros for
            // its grad: its x then adds zeros, or the NaN that it added itself.
            constexpr int kPieces = 2 * F;
            const auto keep = [&](int first, int at, uint8_t *planes, int piece) {
                const int j = piece / 4, h = piece / 2 % 2;
                // the first chunk's number is even: the second one's place differs in one bit
                uint8_t *to = planes + (my_place ^ (h * 16)) + j * 256;
                if (piece % 2 == 0) {
                    *reinterpret_cast<bf16x8 *>(to) =
                        widen8(x[at][j][2 * h], x[at][j][2 * h + 1], f8_step(step[at][j]));
                    return;
                }
                const uint32_t there = first + my_row < count ? 0xffffffffu : 0u;
                typename Pack<T>::V packs[8 / Pack<T>::kN];
#pragma unroll
                for (int q = 0; q < 8 / Pack<T>::kN; ++q) {
                    const int k = h * 8 / Pack<T>::kN + q;
                    packs[q] = g[at][j][k];
                    if constexpr (CUT) packs[q] = end_pack<T>(packs[q], n0 + j * 128 + my_col + k * Pack<T>::kN, a.cols);
                }
                bf16x8 s[P];
                split8<P>(packs, s);
#pragma unroll
                for (int q = 0; q < P; ++q)
                    *reinterpret_cast<u32x4 *>(to + (1 + q) * kPlaneBytes) = __builtin_bit_cast(u32x4, s[q]) & there;
            };
            // What this thread kept of x, once more where a block may hold values beyond bfloat16's largest: looked at
            // after the step, not between its products (5% there)
            const auto keep_finite = [&](int at, uint8_t *planes) {
                int most = step[at][0];
#pragma unroll
                for (int j = 1; j < kRuns; ++j) most = most > step[at][j] ? most : step[at][j];
                if (!__ballot(most >= kF8Beyond)) return;
#pragma unroll
                for (int j = 0; j < kRuns; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        auto *to = reinterpret_cast<bf16x8 *>(planes + (my_place ^ (h * 16)) + j * 256);
                        *to = finite8(*to);
                    }
            };
            const auto keep_all = [&](int first, int at, uint8_t *planes) {
#pragma unroll
                for (int piece = 0; piece < kPieces; ++piece) keep(first, at, planes, piece);
                keep_finite(at, planes);
            };
            const auto operand = [&](const uint8_t *plane, int unit, int deep) {
                typedef __attribute__((address_space(3))) s16x4 *LdsPtr;
                typedef short s16x8 __attribute__((ext_vector_type(8)));
                // of 16 columns each; the unit's number is even: its place is that of the first two, moved
                const uint8_t *at = plane + deep * (kTile * 2) + (from ^ (unit * 32));
                const s16x4 low = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at));
                const s16x4 high = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(at + 4 * (kTile * 2)));
                const s16x8 both = __builtin_shufflevector(low, high, 0, 1, 2, 3, 4, 5, 6, 7);
                return __builtin_bit_cast(bf16x8, both);
            };
            // A step is 2 P phases: 16 rows and one plane of grad each, the smallest plane first. Operand r of a phase: the
            // plane's, and where the rows are new x's.
            constexpr int kPhases = 2 * P;
            constexpr auto operands = [](int phase) { return phase % P == 0 ? 2 * F : F; };
            const auto fetch = [&](const uint8_t *planes, int phase, int r) {
                const int deep = phase / P * 16, q = P - 1 - phase % P;
                if (r < F) n[phase % 2][r] = operand(planes + (1 + q) * kPlaneBytes, wc * 2 * F + r * 2, deep);
                else d[phase / P % 2][r - F] = operand(planes, wr * 2 * F + (r - F) * 2, deep);
            };
            const auto fetch_all = [&](const uint8_t *planes, int phase) {
#pragma unroll
                for (int r = 0; r < operands(phase); ++r) fetch(planes, phase, r);
            };
            // One step, whose first operands are there. Between its products, in this order: the reads of the next phase's
            // operands, the loads of the rows kAhead + 1 steps on, and the rows kAhead steps on to LDS.
            const auto work = [&](int first, int at, const uint8_t *now, const uint8_t *next, uint8_t *after) {
                constexpr int M = F * F;
                __syncthreads();
                if constexpr (kAhead == 1) fetch_all(now, 0);
                unrolled<kPhases * M>([&](auto turn) {
                    constexpr int phase = turn / M, m = turn % M, i = m / F, k = m % F;
                    constexpr bool last = phase + 1 == kPhases;
                    constexpr int reads = !last ? operands(phase + 1) : kAhead == 2 ? operands(0) : 0;
                    // the reads end early enough to be done at the next phase
#pragma unroll
                    for (int r = m * reads * 4 / (M * 3); r < (m + 1) * reads * 4 / (M * 3) && r < reads; ++r)
                        fetch(last ? next : now, last ? 0 : phase + 1, r);
                    acc[i][k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d[phase / P % 2][i], n[phase % 2][k], acc[i][k],
                                                                        0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (phase == 0 && m % (M / 4) == 0 && m / (M / 4) < kRuns) load(1 - at, m / (M / 4));
                    if (phase == 0 && m == M * 3 / 4) seek(first + (kAhead + 2) * kDeep);
                    if (last)
#pragma unroll
                        for (int piece = m * kPieces / M; piece < (m + 1) * kPieces / M; ++piece)
                            keep(first + kAhead * kDeep, at, after, piece);
                });
                keep_finite(at, after);
            };
            load_all(kDeep, 0);
            load_all(2 * kDeep, 1);
            keep_all(0, 0, s_planes);
            if constexpr (kAhead == 2) {
                load_all(3 * kDeep, 0);
                keep_all(kDeep, 1, s_planes + kBytes);
                __syncthreads();
                fetch_all(s_planes, 0);
            }
            // so many steps a turn that registers two deep and LDS kAhead + 1 deep are then the same in every turn
            constexpr int kSteps = kAhead == 2 ? 6 : 2;
            for (int first = 0; first < count;) {
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    constexpr int kPlaces = kAhead + 1;
                    work(first, (u + kAhead) % 2, s_planes + u % kPlaces * kBytes,
                         s_planes + (u + 1) % kPlaces * kBytes, s_planes + (u + kAhead) % kPlaces * kBytes);
                    first += kDeep;
                    if (first >= count) break;
                }
            }
        }
        float *out = a.out + (a.parted ? item : run.expert) * static_cast<int64_t>(a.dim) * a.cols;
        // one pointer that walks the lane's results, so that no address is kept from before
        const int n1 = n0 + wc * F * 32 + lane % 32, d1 = d0 + wr * F * 32 + lane / 32 * 4;
        float *to = out + static_cast<int64_t>(d1) * a.cols + n1;
        const bool inside = a.dim - d0 >= kTile && a.cols - n0 >= kTile;
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int g = 0; g < 16; ++g) {
                const int d = d1 + i * 32 + g / 4 * 8 + g % 4;
#pragma unroll
                for (int k = 0; k < F; ++k)
                    if (inside || (d < a.dim && n1 + k * 32 < a.cols))
                        to[k * 32] = acc[i][k][g];
                to += (g % 4 == 3 ? 5 : 1) * static_cast<int64_t>(a.cols);
                asm volatile("" : "+v"(to));
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
        int64_t k = 0;
        for (; k + 8 <= count; k += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = from[(k + j) * size];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        for (; k < count; ++k) s += from[k * size];
        out[expert * size + i] = s;
    }
}

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int kMaxExperts = 4096;

// Rows of a part and the parts that there can be; one part an expert where its tiles alone fill the chip.
struct Parts {
    int64_t chunk, items;
    int tile;
    bool parted;
};
inline int64_t tiles_of(int64_t dim, int64_t cols, int tile) {
    return ((dim + tile - 1) / tile) * ((cols + tile - 1) / tile);
}
Parts parts_for(int64_t rows, int experts, int64_t dim, int64_t cols) {
    const int64_t all = rows > 0 ? rows : 1;
    // Large tiles, one a unit: 8 x 1024 rows 1024 x 2048 52 us, by small ones 60, 8 x 2048 rows 86 and 104, but 8 x 256
    // rows 30 and 26. With less than a tile a unit they leave units idle: 8192 rows 4096 x 2048 232 and 180.
    const int64_t large = experts * tiles_of(dim, cols, kLarge);
    if (cols >= 8 && (large >= 2 * kUnits || (large >= kUnits && rows >= 768 * static_cast<int64_t>(experts))))
        return {all, experts, kLarge, false};
    const int64_t tiles = tiles_of(dim, cols, kSmall);
    // the parts' tiles fill the chip once (two workgroups a unit), each expert's last part being a shorter one; twice
    // where that leaves fewer parts than experts
    int64_t want = 2 * kUnits / tiles - experts;
    if (want < experts) want = 4 * kUnits / tiles - experts;
    int64_t chunk = want > 0 ? (rows + want - 1) / want : rows;
    chunk = (chunk + kDeep - 1) / kDeep * kDeep;
    chunk = chunk < 8 * kDeep ? 8 * kDeep : chunk;
    if (experts * tiles >= 2 * kUnits || chunk >= rows) return {all, experts, kSmall, false};
    return {chunk, rows / chunk + experts, kSmall, true};
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
    const int64_t tiles = parts.items * tiles_of(dim, cols, parts.tile);
    const int64_t whole = (tiles + kDies - 1) / kDies * kDies, most = 1 << 20;
    const dim3 grid(static_cast<unsigned>(whole < most ? whole : most));
#define GS_WEIGHT_GRAD_F(T, F, CUT, NARROW)                                                                           \
    hipLaunchKernelGGL((weight_grad_kernel<T, F, CUT, NARROW>), grid, dim3(kThreads), 0, stream, a, parts.items)
#define GS_WEIGHT_GRAD(T)                                                                  \
    do {                                                                                   \
        if (cols < Pack<T>::kN) GS_WEIGHT_GRAD_F(T, 2, false, true);                       \
        else if (cols % Pack<T>::kN != 0 && parts.tile == kLarge) GS_WEIGHT_GRAD_F(T, 4, true, false); \
        else if (cols % Pack<T>::kN != 0) GS_WEIGHT_GRAD_F(T, 2, true, false);             \
        else if (parts.tile == kLarge) GS_WEIGHT_GRAD_F(T, 4, false, false);               \
        else GS_WEIGHT_GRAD_F(T, 2, false, false);                                         \
    } while (0)
    if (dtype == GS_F32) GS_WEIGHT_GRAD(float);
    else if (dtype == GS_BF16) GS_WEIGHT_GRAD(__bf16);
    else GS_WEIGHT_GRAD(_Float16);
#undef GS_WEIGHT_GRAD
#undef GS_WEIGHT_GRAD_F
    GS_LAUNCH_TRY("weight_grad_kernel");
    if (parts.parted) {
        const int64_t groups = (dim * cols + kThreads - 1) / kThreads, joins = groups * experts;
        hipLaunchKernelGGL(weight_grad_join_kernel, dim3(static_cast<unsigned>(joins < most ? joins : most)),
                           dim3(kThreads), 0, stream, a, static_cast<const float *>(workspace), parts.items, groups, out);
        GS_LAUNCH_TRY("weight_grad_join_kernel");
    }
    return ok();
}
