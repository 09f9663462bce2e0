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
// to y = |x| * 2^(7 - byte), whose exponent field is then e4m3's (bits below
// fp32's least subnormal dropped), the code is (bits(y) + r) >> 20 for a 20-bit
// r, subnormal codes included. r uniform is stochastic rounding. gfx950
// converts so in one instruction (scale, add the seed's high 20 bits, cut,
// place the byte), to nearest even in another, and back in a third; the GPU
// tests compare all three with this formula: decoding for every code and scale,
// encoding over every exponent of a block, subnormal codes included.
//
// Why stochastic. With beta2 = 0.999 the second moment moves by about 0.1% a
// step, against code steps of 6-12%: rounding to nearest would return the old
// code for ever. The stochastic rounding moves it by one code now and then and
// keeps its mean right, at the least code and above.
//
// A positive second moment never rounds to zero (its code is at least 1): with
// v = 0 beside a surviving m, m / (sqrt(v) + eps) would be a step of m / eps. The
// price: a v below the least code, 2^-17 to 2^-16 of its block's largest, reads
// as that code while the block's scale stays, and its element's steps are smaller
// by the root of the ratio.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "zero_mi355x.h"

namespace zero {
namespace state8 {

constexpr int kBlock = ZERO_STATE8_BLOCK;
static_assert(kBlock == 128, "the lane groups below are laid out for blocks of 128");

inline int64_t blocks_of(int64_t n) { return n / kBlock + (n % kBlock != 0); }

// ------------------------------------------------------------ random words
//
// Element i (of the caller's numbering) of step t draws one 32-bit word from
// (seed, t, i) alone, so results depend on no launch shape, and a shard cut
// into pieces rounds as the whole does. The numbering is cut into windows of
// 2^28 elements. A window's key in a step is a 64-bit multiply-and-shift mix of
// (seed, t, window); the 8 elements of a group share two words a and b (b odd)
// mixed from the group's index in its window and the key, and element j of the
// group has a + j * b: one addition per element. b follows from a, so a group
// has 32 bits of state, and its words are an arithmetic progression modulo 2^32
// with an odd difference. The first moment takes the word's high 20 bits, the
// second its low 20. The multipliers are the fractional bits of square roots of
// primes (made odd).
//
// Why windows. The group's mix is short: a high bit of the index reaches few
// bits of the word, so with one key for all elements the draws of two of them
// 2^28 or more apart were correlated in every step: over many pairs by 0.01 at
// 2^28 and 0.1 at 2^32, some pairs by 0.86. With keys of their own no correlation
// is found at 2^28 to 2^40; within a window it stays below 0.015 (2^27 apart).
constexpr int kWindowBits = 28;
constexpr uint32_t kWindowGroups = 1u << (kWindowBits - 3);

struct Key {
    uint32_t k0, k1;
};

// A step's part of its windows' keys.
__host__ __device__ inline uint64_t step_base(uint64_t seed, uint64_t step) {
    return seed + step * 0x6A09E667F3BCC909ull;
}

__host__ __device__ inline Key window_key(uint64_t base, uint64_t window) {
    uint64_t z = base + window * 0xA54FF53A5F1D36F1ull;
    z = (z ^ (z >> 32)) * 0xBB67AE8584CAA73Bull;
    z = (z ^ (z >> 29)) * 0x3C6EF372FE94F82Bull;
    z ^= z >> 32;
    return Key{static_cast<uint32_t>(z), static_cast<uint32_t>(z >> 32)};
}

struct Words {
    uint32_t a, b;
};

// group: its index in its window.
__device__ __forceinline__ Words group_words(uint32_t group, Key key) {
    uint32_t x = (group ^ key.k0) * 0xA54FF53Bu;
    x ^= x >> 16;
    x = (x + key.k1) * 0x510E527Fu;
    x ^= x >> 15;
    uint32_t b = x * 0x9B05688Du;
    b = (b ^ (b >> 16)) | 1u;
    return Words{x, b};
}

// The words of the group that holds element start + t. start is a multiple of
// the block and the same in every lane, t below `span`, so that the lanes lie in
// one window or, seldom, on both sides of a border.
__device__ __forceinline__ Words words_at(int64_t start, uint32_t t, uint32_t span, uint64_t base) {
    const uint64_t window = static_cast<uint64_t>(start) >> kWindowBits;
    const uint32_t at = static_cast<uint32_t>(start >> 3) & (kWindowGroups - 1u);
    const uint32_t group = at + (t >> 3);
    const Key key = window_key(base, window);
    if (at + span / 8u <= kWindowGroups) return group_words(group, key);     // the same in every lane
    const Key next = window_key(base, window + 1);
    return group < kWindowGroups ? group_words(group, key) : group_words(group - kWindowGroups, next);
}

// ------------------------------------------------------------ block maximum

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), kCtrl, 0xF, 0xF, false));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

constexpr int kLaneElems = 4;      // consecutive elements a lane holds in every kernel here

// The largest x over the 32 lanes that hold one block (4 elements a lane, the
// wave's lanes in order), in every one of them. All lanes take part. Rows of 16
// lanes by rotations within the row, then one swap of neighbouring rows.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    x = umax(x, dpp<0x128>(x));     // row_ror:8
    x = umax(x, dpp<0x124>(x));     // row_ror:4
    x = umax(x, dpp<0x122>(x));     // row_ror:2
    x = umax(x, dpp<0x121>(x));     // row_ror:1
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return umax(s[0], s[1]);
}

// The bits of the largest magnitude of four values; a NaN wins (the IEEE
// maximum, one v_maximum3 per two values).
__device__ __forceinline__ uint32_t max_bits4(const float (&x)[4]) {
    float m = __builtin_elementwise_maximum(__builtin_fabsf(x[0]), __builtin_fabsf(x[1]));
    m = __builtin_elementwise_maximum(m, __builtin_fabsf(x[2]));
    m = __builtin_elementwise_maximum(m, __builtin_fabsf(x[3]));
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
    const uint32_t field = max_bits >> 23;
    return field == 255u ? 255u : (field > 7u ? field - 7u : 0u);
}

// ------------------------------------------------------------ codes

// The scale as the conversions take it: the power of two in an fp32's exponent
// field (byte 0 stands for 2^-127 there, byte 255 for NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four codes as fp32 (in a block with this scale byte).
__device__ __forceinline__ void decode4(uint32_t word, uint32_t byte, float (&out)[4]) {
    const float s = scale_of(byte);
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, s, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, s, true);
    out[0] = lo[0];
    out[1] = lo[1];
    out[2] = hi[0];
    out[3] = hi[1];
}

// Four elements stochastically rounded with the high 20 bits of r[0..3], as one
// word; zeros in a block that is not finite.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], uint32_t byte, const uint32_t (&r)[4]) {
    const float s = scale_of(byte);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[0], r[0], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[1], r[1], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[2], r[2], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[3], r[3], s, 3);
    return byte == 255u ? 0u : w;
}

// The same, rounded to nearest even.
__device__ __forceinline__ uint32_t nearest4(const float (&x)[4], uint32_t byte) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float s = scale_of(byte);
    s16x2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], s, true);
    return byte == 255u ? 0u : __builtin_bit_cast(uint32_t, w);
}

// Raises the zero codes of positive elements to 1 (second moments), in a block
// with a finite scale. Zero codes are rare (the element is below 2^-16 of its
// block's largest, or zero), so one test of the word decides for the four.
__device__ __forceinline__ uint32_t positive4(uint32_t w, const float (&x)[4], uint32_t byte) {
    if (((w - 0x01010101u) & ~w & 0x80808080u) != 0u && byte != 255u) {      // a zero byte
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (((w >> (8 * k)) & 0xFFu) == 0u && x[k] > 0.0f) w |= 1u << (8 * k);
    }
    return w;
}

}  // namespace state8
}  // namespace zero
