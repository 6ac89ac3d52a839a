// 8-bit values on gfx950: e4m3 (OCP: 448 the largest, no infinity) with a scale 2^(byte - 127) for each block of 128 along
// a row. Rows are padded to whole blocks with zeros, so a block is always 128 bytes at a multiple of 16.
#pragma once

#include "gs_types.hpp"

namespace gs {

constexpr int kF8Block = 128;
constexpr int kF8Bias = 127;

__host__ __device__ constexpr int64_t f8_blocks(int64_t dim) { return (dim + kF8Block - 1) / kF8Block; }

// The scale's byte for a block whose largest finite magnitude has these bits: the least e with amax <= 448 * 2^e, within
// [-126, 127]; 0 for a block of zeros. 448 is 1.75 * 2^8.
__device__ __forceinline__ int f8_scale(uint32_t amax_bits) {
    if (amax_bits == 0) return kF8Bias;
    // adding a quarter less one unit carries into the exponent where the fraction is above 1.75
    const int byte = static_cast<int>((amax_bits + 0x1fffffu) >> 23) - 8;
    return byte < 1 ? 1 : byte;  // at most 254 + 1 - 8
}
// 2^(byte - 127) and its inverse; byte in [1, 253].
__device__ __forceinline__ float f8_step(int byte) { return __builtin_bit_cast(float, static_cast<uint32_t>(byte) << 23); }
__device__ __forceinline__ float f8_inverse(int byte) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(254 - byte) << 23);
}

// The bits of a finite magnitude, 0 for infinities and NaN: they leave the scale to the rest of the block.
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

// Four values times `inverse` as e4m3, nearest and to even; infinities become NaN, as e4m3 has none.
__device__ __forceinline__ uint32_t f8_pack(float a, float b, float c, float d, float inverse) {
    const auto scaled = [&](float v) {
        return finite_bits(v) != 0 || v == 0.0f ? v * inverse : __builtin_nanf("");
    };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(a), scaled(b), 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(scaled(c), scaled(d), w, true));
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 held values as bfloat16. That loses nothing (e4m3 has 4 bits and the scale none) of multiples of 2^-133, which those of
// scale bytes from 3 on are; smaller multiples are rounded to one of 2^-133. From kF8Beyond on a value may be beyond
// bfloat16's largest: rounding up makes one of a finite value next to it.
constexpr int kF8Beyond = 247;
__device__ __forceinline__ bf16x8 widen8(uint32_t first, uint32_t second, float step) {
    bf16x8 out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? first : second;
        const bf16x2 two = k % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, step, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, step, false);
        out[2 * k] = two[0];
        out[2 * k + 1] = two[1];
    }
    return out;
}

// The largest in place of infinities, as where a value is restored: an infinity would make NaN of every zero that it meets.
// NaN stays.
__device__ __forceinline__ bf16x8 finite8(bf16x8 v) {
    u32x4 bits = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if ((bits[k] & 0x7fffu) == 0x7f80u) --bits[k];
        if ((bits[k] & 0x7fff0000u) == 0x7f800000u) bits[k] -= 0x10000u;
    }
    return __builtin_bit_cast(bf16x8, bits);
}

}  // namespace gs
