// Element types of the training operators (layer norm, experts, orthogonalised updates): 16-byte loads and stores
// of rows that start at any element, and conversions to and from float32.
#pragma once

#include <initializer_list>

#include "gs_internal.hpp"

namespace gs {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Pack {
    static constexpr int kN = 16 / sizeof(T);  // elements of one 16-byte load
    typedef T V __attribute__((ext_vector_type(kN)));
    // Rows of an odd width start at any multiple of the element's size, and gfx950's vector memory takes a
    // 16-byte access at any address, so one path serves every alignment.
    typedef V VU __attribute__((aligned(sizeof(T))));
};

// Columns [col, col + kN) of a row of `dim` elements, those past the end 0.
template <typename T>
__device__ __forceinline__ typename Pack<T>::V load_pack(const T *__restrict__ row, int64_t col, int64_t dim) {
    if (col + Pack<T>::kN <= dim) return *reinterpret_cast<const typename Pack<T>::VU *>(row + col);
    typename Pack<T>::V v;
#pragma unroll
    for (int j = 0; j < Pack<T>::kN; ++j) v[j] = col + j < dim ? row[col + j] : static_cast<T>(0.0f);
    return v;
}

// The same for rows of a pack at least, in two parts. A pack that the row's end cuts, or that lies past it, is read to end
// with the row, so that every lane's load is the same and none waits; end_pack, where the values are first needed,
// shifts it to its place. Rows of whole packs (a uniform branch) skip that. ONCE: read this one time, and kept from
// taking room in the caches.
template <bool ONCE = false, typename T>
__device__ __forceinline__ typename Pack<T>::V read_pack(const T *__restrict__ row, int col, int dim) {
    const int last = dim - Pack<T>::kN;
    const auto *from = reinterpret_cast<const typename Pack<T>::VU *>(row + (col < last ? col : last));
    return ONCE ? __builtin_nontemporal_load(from) : *from;
}
template <typename T>
__device__ __forceinline__ typename Pack<T>::V end_pack(typename Pack<T>::V v, int col, int dim) {
    constexpr int N = Pack<T>::kN;
    if (dim % N != 0) {
        int past = col - (dim - N);
        past = past < 0 ? 0 : past > N ? N : past;
        unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, v);
        bits = past < N ? bits >> (past * 8 * static_cast<int>(sizeof(T))) : static_cast<unsigned __int128>(0);
        return __builtin_bit_cast(typename Pack<T>::V, bits);
    }
    if (col >= dim) v = static_cast<T>(0.0f);
    return v;
}

template <typename T>
__device__ __forceinline__ void store_pack(T *__restrict__ row, int64_t col, int64_t dim, typename Pack<T>::V v) {
    if (col + Pack<T>::kN <= dim) {
        *reinterpret_cast<typename Pack<T>::VU *>(row + col) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < Pack<T>::kN; ++j)
        if (col + j < dim) row[col + j] = v[j];
}

// N consecutive values of an array of T at col as float32 (0 past the end), whole packs.
template <int N, typename T>
__device__ __forceinline__ void load_floats(const T *__restrict__ row, int64_t col, int64_t dim, float *out) {
    constexpr int P = Pack<T>::kN;
    static_assert(N % P == 0, "whole packs");
#pragma unroll
    for (int i = 0; i < N / P; ++i) {
        const typename Pack<T>::V v = load_pack(row, col + i * P, dim);
#pragma unroll
        for (int j = 0; j < P; ++j) out[i * P + j] = static_cast<float>(v[j]);
    }
}

// The same for rows of a pack at least.
template <int N, typename T>
__device__ __forceinline__ void load_floats_long(const T *__restrict__ row, int col, int dim, float *out) {
    constexpr int P = Pack<T>::kN;
    static_assert(N % P == 0, "whole packs");
    typename Pack<T>::V v[N / P];
#pragma unroll
    for (int i = 0; i < N / P; ++i) v[i] = read_pack(row, col + i * P, dim);
#pragma unroll
    for (int i = 0; i < N / P; ++i) {
        v[i] = end_pack<T>(v[i], col + i * P, dim);
#pragma unroll
        for (int j = 0; j < P; ++j) out[i * P + j] = static_cast<float>(v[i][j]);
    }
}

// Sum over the lanes of a group of G consecutive lanes (G a power of two up to 64), in every lane.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// An argument's bytes; none: an argument that is not given.
struct Span {
    const char *name;
    const void *at;
    size_t bytes;
};

// Refuses outputs (a workspace among them) that overlap an input or each other: the kernels read and write them in any
// order, and a count that changes between two reads would lead a store out of its array.
inline gs_status check_apart(const char *name, std::initializer_list<Span> outputs,
                             std::initializer_list<Span> inputs) {
    const auto apart = [](const Span &a, const Span &b) {
        if (!a.at || !b.at || a.bytes == 0 || b.bytes == 0) return true;
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
        return x < y ? y - x >= a.bytes : x - y >= b.bytes;
    };
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (!apart(*o, i)) return fail(GS_ERR_INVALID_ARG, "%s: %s overlaps %s", name, o->name, i.name);
        for (const Span *p = outputs.begin(); p != o; ++p)
            if (!apart(*o, *p)) return fail(GS_ERR_INVALID_ARG, "%s: %s overlaps %s", name, o->name, p->name);
    }
    return GS_OK;
}

inline bool known_dtype(int dtype) { return dtype == GS_F32 || dtype == GS_BF16 || dtype == GS_F16; }
inline size_t dtype_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

}  // namespace gs
