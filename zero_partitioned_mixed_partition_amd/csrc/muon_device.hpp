// Device pieces that the Muon kernels share: a call's matrices, and reading and
// writing the caller's arrays.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_common.hpp"
#include "muon_plan.hpp"

#pragma clang fp contract(off)

namespace zero {
namespace muon {
namespace dev {

typedef _Float16 f16;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

// The matrices of one call: a device table of descriptors, or (table NULL) a stack of equal matrices described by its
// first.
struct Matrices {
    const Desc* table;
    const uint32_t* index[kGrids];    // per grid, the descriptor of each workgroup
    Desc base;
    int64_t src_bytes;            // from one matrix of a stack to the next
    int64_t numel;
    int64_t area;
    int64_t square_tile, rect_tile;    // of the products of square matrices, and of those with X's shape
    uint32_t per[kGrids];         // workgroups of one matrix of a stack, per grid
    uint32_t total[kGrids];
    double* partials;
    float* kappa;
    char* ws;
    uint32_t matrices;
    int32_t side;                 // 64, 96 or 128 where every short side is at most that, else 0
    int64_t short_area;
    int32_t* part_exponent;
    struct ShortScale* short_scale;
};

// A matrix's power of two and factor, from the sum over its parts: X is factor * 2^(13 - exponent) times the matrix.
struct ShortScale {
    int32_t exponent;
    float factor;
};

// Matrix i.
__device__ __forceinline__ Desc matrix(const Matrices& m, uint32_t i) {
    if (m.table != nullptr) return m.table[i];
    Desc d = m.base;
    const int64_t at = m.numel * i;
    d.src = static_cast<const char*>(d.src) + m.src_bytes * i;
    if (d.momentum != nullptr) d.momentum += at;
    if (d.master != nullptr) d.master += at;
    d.out += at;
    d.ws += m.area * i;
    d.short_ws += m.short_area * i;
    d.first_partial = d.chunks * static_cast<int32_t>(i);
    d.first[kByPart] = d.parts * static_cast<int32_t>(i);
    d.id = static_cast<int32_t>(i);
    return d;
}

// The matrix of workgroup t of a grid, and the workgroup's number within it.
__device__ __forceinline__ Desc find(const Matrices& m, int grid, uint32_t t, uint32_t* local) {
    if (m.table != nullptr) {
        const Desc d = m.table[m.index[grid][t]];
        *local = t - static_cast<uint32_t>(d.first[grid]);
        return d;
    }
    const uint32_t i = t / m.per[grid];
    *local = t - i * m.per[grid];
    return matrix(m, i);
}

// Four values as two fp16 parts each, hi + lo (22 bits). They go through registers of their own: the compiler may otherwise
// fold the product that a value is into one of the two conversions to hi (the stored one and the subtracted one), which
// then round apart now and then.
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, f16x4* hi, f16x4* lo) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    asm("" : "+v"(x0), "+v"(x1), "+v"(x2), "+v"(x3));
    const f16x2 a = __builtin_convertvector((f32x2{x0, x1}), f16x2), b = __builtin_convertvector((f32x2{x2, x3}), f16x2);
    const f16x2 c = __builtin_convertvector((f32x2{x0 - static_cast<float>(a.x), x1 - static_cast<float>(a.y)}), f16x2),
                d = __builtin_convertvector((f32x2{x2 - static_cast<float>(b.x), x3 - static_cast<float>(b.y)}), f16x2);
    *hi = f16x4{a.x, a.y, b.x, b.y};
    *lo = f16x4{c.x, c.y, d.x, d.y};
}

// What the momentum pass computes per element.
struct MomentumScalars {
    float mu;
    int32_t nesterov;
    const float* clip;            // NULL: 1
};

__device__ __forceinline__ bool skipped(const float* clip) { return clip != nullptr && !isfinite(*clip); }

// Four consecutive values; the arrays are aligned to their elements only.
struct __attribute__((packed, aligned(4))) F32x4 {
    float v[4];
};
struct __attribute__((packed, aligned(2))) U16x4 {
    uint16_t v[4];
};

// Reads n <= 4 values at element i as fp32 (the rest 0), four at once where n is 4.
__device__ __forceinline__ void read4(const float* p, int64_t i, int n, float* out) {
    if (n == 4) {
        const F32x4 x = *reinterpret_cast<const F32x4*>(p + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = x.v[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = k < n ? p[i + k] : 0.0f;
    }
}
__device__ __forceinline__ void read4(const uint16_t* p, int64_t i, int n, float* out) {
    if (n == 4) {
        const U16x4 x = *reinterpret_cast<const U16x4*>(p + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = ::zero::dev::bf16_to_f32(x.v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = k < n ? ::zero::dev::bf16_to_f32(p[i + k]) : 0.0f;
    }
}

// Writes n <= 4 values at element i, four at once where n is 4.
__device__ __forceinline__ void write4(float* p, int64_t i, int n, const float* v) {
    if (n == 4) {
        *reinterpret_cast<F32x4*>(p + i) = F32x4{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) p[i + k] = v[k];
    }
}
__device__ __forceinline__ void write4(uint16_t* p, int64_t i, int n, const uint16_t* v) {
    if (n == 4) {
        *reinterpret_cast<U16x4*>(p + i) = U16x4{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) p[i + k] = v[k];
    }
}

// The matrix to orthogonalise at elements i to i + n - 1. kSource: 0 bf16, 1 fp32, 2 momentum and gradient (kUpdate:
// the momentum is moved on and written first).
template <int kSource, bool kUpdate>
__device__ __forceinline__ void input4(const Desc& d, int64_t i, int n, const MomentumScalars& s, float clip, float* u) {
    if constexpr (kSource == 0) read4(static_cast<const uint16_t*>(d.src), i, n, u);
    if constexpr (kSource == 1) read4(static_cast<const float*>(d.src), i, n, u);
    if constexpr (kSource == 2) {
        float buf[4], g[4] = {};
        read4(d.momentum, i, n, buf);
        if (kUpdate || s.nesterov) read4(static_cast<const uint16_t*>(d.src), i, n, g);
        if constexpr (kUpdate) {
#pragma unroll
            for (int k = 0; k < 4; ++k) buf[k] = s.mu * buf[k] + g[k] * clip;
            write4(d.momentum, i, n, buf);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = s.nesterov ? g[k] * clip + s.mu * buf[k] : buf[k];
    }
}

// The weight update of the last product's epilogue.
struct Update {
    double lr;
    float decay;                  // 1 - lr * weight_decay
    const float* clip;
};

// The last step of `here` <= 8 elements from element `first` on: the orthogonalised values' bf16 bits o to the caller
// (kEnd 1), or the weight update with them (kEnd 2; w: the master's values there).
template <int kEnd>
__device__ __forceinline__ void finish8(const Desc& d, const Update& u, float rate, int64_t first, int here, const uint16_t* o,
                                        float* w) {
    uint16_t bits[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (kEnd == 1) {
            bits[k] = o[k];
        } else {
            w[k] = w[k] * u.decay;
            w[k] = w[k] - rate * ::zero::dev::bf16_to_f32(o[k]);
            bits[k] = static_cast<uint16_t>(::zero::dev::f32_to_bf16(w[k]));
        }
    }
    if constexpr (kEnd == 2) {
        write4(d.master, first, here < 4 ? here : 4, w);
        write4(d.master, first + 4, here < 4 ? 0 : here - 4, w + 4);
    }
    write4(d.out, first, here < 4 ? here : 4, bits);
    write4(d.out, first + 4, here < 4 ? 0 : here - 4, bits + 4);
}

// The four values of one column in each lane of a quad (two in each word), as one row's four columns in each.
__device__ __forceinline__ f16x4 quad_transpose(f16x4 v) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    u32x2_t w = __builtin_bit_cast(u32x2_t, v);
    const uint32_t lane = threadIdx.x;
    // lanes 2k and 2k + 1: (r0 r1 | r2 r3) of two columns -> rows 0 / 1 and 2 / 3 of both
    const bool odd = lane & 1;
    // what the neighbour needs of this lane: an even lane's odd rows, an odd lane's even rows
    const uint32_t give = odd ? __builtin_amdgcn_perm(w.y, w.x, 0x05040100) : __builtin_amdgcn_perm(w.y, w.x, 0x07060302);
    const uint32_t keep = odd ? __builtin_amdgcn_perm(w.y, w.x, 0x07060302) : __builtin_amdgcn_perm(w.y, w.x, 0x05040100);
    const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);       // quad_perm 1 0 3 2
    // keep: this lane's rows (0, 2) or (1, 3); got: the neighbour's same rows. Columns in order: even lane first.
    const uint32_t left = odd ? got : keep, right = odd ? keep : got;
    uint32_t a = __builtin_amdgcn_perm(right, left, 0x05040100);     // row 0 (1), two columns
    uint32_t b = __builtin_amdgcn_perm(right, left, 0x07060302);     // row 2 (3)
    // lanes q and q ^ 2: row 0 (1) stays in lanes 0, 1; row 2 (3) goes to lanes 2, 3
    const bool high = lane & 2;
    const uint32_t give2 = high ? a : b;
    const uint32_t got2 = __builtin_amdgcn_mov_dpp(give2, 0x4E, 0xF, 0xF, true);     // quad_perm 2 3 0 1
    u32x2_t out;
    out.x = high ? got2 : a;
    out.y = high ? b : got2;
    return __builtin_bit_cast(f16x4, out);
}

}  // namespace dev
}  // namespace muon
}  // namespace zero
