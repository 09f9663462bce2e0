// Optimizer moments held in 8 bits: blocks of 128 consecutive elements, an
// OCP e4m3 code per element and one power-of-two scale byte per block (e8m0),
// value = e4m3(code) * 2^(byte - 127). Shared by the 8-bit AdamW kernels and
// the conversions to and from fp32.
//
// "Zero Redundancy Optimizer (ZeRO) and Fully Sharded Data Parallelism (FSDP):
// Mathematical Foundations ...", section "Static Memory Allocation" (the first
// and second moments m_t and v_t are two thirds of the optimizer state).
//
// Scale. A block's byte follows from the exponent field E of its largest
// magnitude: max(E - 7, 0), so that this magnitude lies in [2^7, 2^8) in code
// units. e4m3 ends at 448: rounding up reaches 2^8 at most and never
// saturates. A power of two costs a floating-point code no precision, its
// division is exact, and the byte is 1/4 of an fp32 scale. A block holding an
// infinity or NaN has byte 255 (e8m0's NaN) and zero codes: it reads as NaN.
//
// Code. e4m3 (4 exponent bits, 3 mantissa bits, gradual underflow) is fp32
// with the low exponents 0..15 and the mantissa cut to 3 bits: with |x| scaled
// to y = |x| * 2^(7 - byte), whose exponent field is then e4m3's, the code is
// (bits(y) + r) >> 20 for a 20-bit r, subnormal codes included (y is then a
// subnormal fp32). r uniform gives stochastic rounding, E[value] = x exactly
// where y is normal; r = 0x7FFFF + (bit 20) gives round to nearest even.
//
// Why stochastic. With beta2 = 0.999 the second moment moves by about 0.1% a
// step, against code steps of 6-12%: rounding to nearest would return the old
// code for ever. The stochastic rounding moves it by one code now and then and
// keeps its mean right.
//
// A positive second moment never rounds to zero (its code is at least 1): with
// v = 0 beside a surviving m, m / (sqrt(v) + eps) would be a step of m / eps.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "zero_mi355x.h"

namespace zero {
namespace state8 {

constexpr int kBlock = ZERO_STATE8_BLOCK;
static_assert(kBlock == 128, "the lane groups below are laid out for blocks of 128");

inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// ------------------------------------------------------------ random words
//
// Element i (of the caller's numbering) of step t draws one 32-bit word from
// (seed, t, i) alone, so results depend on no launch shape, and a shard cut
// into windows rounds as the whole does. A step's key is a 64-bit
// multiply-and-shift mix of (seed, t); the 8 elements of a group share two
// words a and b (b odd) mixed from the group's index and the key, and element
// j of the group has a + j * b: one addition per element, and any two of the 8
// are independent but for the low two bits. The first moment takes the word's
// high 20 bits, the second its low 20. The multipliers are the fractional bits
// of square roots of primes (made odd).
struct Key {
    uint32_t k0, k1;
};

__host__ __device__ inline Key step_key(uint64_t seed, uint64_t step) {
    uint64_t z = seed + step * 0x6A09E667F3BCC909ull;
    z = (z ^ (z >> 32)) * 0xBB67AE8584CAA73Bull;
    z = (z ^ (z >> 29)) * 0x3C6EF372FE94F82Bull;
    z ^= z >> 32;
    return Key{static_cast<uint32_t>(z), static_cast<uint32_t>(z >> 32)};
}

struct Words {
    uint32_t a, b;
};

__device__ __forceinline__ Words group_words(uint64_t group, Key key) {
    uint32_t x = (static_cast<uint32_t>(group) ^ key.k0) * 0xA54FF53Bu;
    x ^= x >> 16;
    x = (x + static_cast<uint32_t>(group >> 32) + key.k1) * 0x510E527Fu;
    x ^= x >> 15;
    uint32_t b = x * 0x9B05688Du;
    b = (b ^ (b >> 16)) | 1u;
    return Words{x, b};
}

// ------------------------------------------------------------ block maximum

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), kCtrl, 0xF, 0xF, false));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest x over the 128 / E lanes that hold one block (E elements a lane,
// the wave's lanes in order), in every one of them. All lanes take part. Rows
// of 16 lanes by rotations within the row; 32 lanes by one swap of row pairs.
template <int E>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    static_assert(E == 4 || E == 8, "16 or 32 lanes a block");
    x = umax(x, dpp<0x128>(x));     // row_ror:8
    x = umax(x, dpp<0x124>(x));     // row_ror:4
    x = umax(x, dpp<0x122>(x));     // row_ror:2
    x = umax(x, dpp<0x121>(x));     // row_ror:1
    if (E == 4) {
        const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = umax(s[0], s[1]);
    }
    return x;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
    const uint32_t field = max_bits >> 23;
    return field == 255u ? 255u : (field > 7u ? field - 7u : 0u);
}

// ------------------------------------------------------------ codes

// Four codes as fp32 (in a block with this scale byte).
__device__ __forceinline__ void decode4(uint32_t word, uint32_t byte, float* out) {
    word = byte == 255u ? 0x7F7F7F7Fu : word;          // e4m3's NaN
    const int e = static_cast<int>(byte) - 127;
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(word), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(word), true);
    out[0] = ldexpf(lo[0], e);
    out[1] = ldexpf(lo[1], e);
    out[2] = ldexpf(hi[0], e);
    out[3] = ldexpf(hi[1], e);
}

// |x| in code units, as the fp32 whose exponent field is e4m3's.
__device__ __forceinline__ uint32_t code_bits(float x, uint32_t byte) {
    return magnitude(ldexpf(x, 7 - static_cast<int>(byte)));
}

// A code in the top byte of a word: t holds the rounded bits(y), whose bit 27
// and above are clear.
__device__ __forceinline__ uint32_t top_code(uint32_t t, float x) {
    return ((t << 4) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u);
}

// The top bytes of four words as one word, the first lowest.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0703u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x07030C0Cu);
    return lo | hi;
}

// Element x of the first moment, stochastically rounded with word r.
__device__ __forceinline__ uint32_t first_code(float x, uint32_t byte, uint32_t r) {
    return top_code(code_bits(x, byte) + (r >> 12), x);
}

// Element x of the second moment: at least code 1 where x is positive.
__device__ __forceinline__ uint32_t second_code(float x, uint32_t byte, uint32_t r) {
    uint32_t t = code_bits(x, byte) + (r & 0xFFFFFu);
    t = umax(t, x > 0.0f ? 1u << 20 : 0u);
    return top_code(t, x);
}

// Element x rounded to nearest even.
__device__ __forceinline__ uint32_t nearest_code(float x, uint32_t byte, bool second) {
    const uint32_t y = code_bits(x, byte);
    uint32_t t = y + 0x7FFFFu + ((y >> 20) & 1u);
    if (second) t = umax(t, x > 0.0f ? 1u << 20 : 0u);
    return top_code(t, x);
}

}  // namespace state8
}  // namespace zero
