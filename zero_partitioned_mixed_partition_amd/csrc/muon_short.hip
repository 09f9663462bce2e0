// Muon on gfx950 for matrices with a short side of at most 128: three launches
// where the tiled products take eighteen.
//
// X X^T is m x m with m <= 128, so every step runs on it alone, in the LDS of
// one workgroup a matrix, and the long side n is passed over twice:
//   gram   the momentum pass, and each part's sum of u u^T
//   chain  A = the parts' sum / |u|^2; per step C = a + b A + c A^2, Q <- C Q,
//          A <- C A C; at the end Q = C_n ... C_1
//   apply  Q X, and the weight update
// Values are two fp16 parts (hi + lo, 22 bits) and a product three MFMAs (the lo
// lo term is below what is kept), so that five steps in a row on A keep 1e-4 of
// the result; with one part the directions of small singular values would be
// lost, since what rounding A leaves there grows by a^2 = 11.9 a step.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "internal.hpp"
#include "muon_device.hpp"
#include "muon_short.hpp"

#pragma clang fp contract(off)

namespace {

using namespace zero::muon;
using namespace zero::muon::dev;

constexpr int kStep = 64;          // of the long side, at a time
constexpr int kEmpty = -4096;      // the exponent of nothing but zeros

// A thread's values of a step along the long side, in blocks of 4 x 4 (rows and columns of the source).
template <int M>
struct Held {
    static constexpr int kBlocks = (4 * M + kThreads - 1) / kThreads;
    float v[kBlocks][4][4];
};

// Calls f(i, down, right) for the thread's blocks: block i covers source rows 4 down and columns 4 right on, counted from
// the step's first; the threads run along the source's rows.
template <int M, typename F>
__device__ __forceinline__ void each_block(bool tall, F f) {
#pragma unroll
    for (int i = 0; i < Held<M>::kBlocks; ++i) {
        const int b = threadIdx.x + i * kThreads, per_row = tall ? M / 4 : kStep / 4;
        if (4 * M % kThreads == 0 || b < 4 * M) f(i, b / per_row, b % per_row);
    }
}

template <int M, int kSource, bool kUpdate>
__device__ __forceinline__ void hold(const Desc& d, bool tall, int32_t at, const MomentumScalars& s, float clip, Held<M>& h) {
    each_block<M>(tall, [&](int i, int down, int right) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t r = (tall ? at : 0) + down * 4 + k, c = (tall ? 0 : at) + right * 4;
            int n = r < d.rows ? d.cols - c : 0;
            n = n < 0 ? 0 : n > 4 ? 4 : n;
            input4<kSource, kUpdate>(d, static_cast<int64_t>(r) * d.cols + c, n, s, clip, h.v[i][k]);
        }
    });
}

// The held values times 2^shift as hi and lo parts, in rows of `ld` at `to` (lo parts kPart values on). kByLong: a row
// for each place of the long side, else of the short one.
template <int M, bool kByLong, bool kLow>
__device__ __forceinline__ void split(const Held<M>& h, bool tall, int shift, int ld, f16* to, int part) {
    each_block<M>(tall, [&](int i, int down, int right) {
        const bool as_held = tall == kByLong;            // the source's rows are the rows wanted
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f16x4 hi, lo;
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = ldexpf(as_held ? h.v[i][k][j] : h.v[i][j][k], shift);
            split4(x[0], x[1], x[2], x[3], &hi, &lo);
            f16* const at = to + ((as_held ? down : right) * 4 + k) * ld + (as_held ? right : down) * 4;
            *reinterpret_cast<f16x4*>(at) = hi;
            if constexpr (kLow) *reinterpret_cast<f16x4*>(at + part) = lo;
        }
    });
}

__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The row, within its 32 x 32 block, of a lane's value k.
__device__ __forceinline__ int block_row(int k) { return k / 4 * 8 + threadIdx.x % 64 / 32 * 4 + k % 4; }

// The momentum pass and u u^T of a part: fp32 sums times 2^(2 (13 - e)), e the part's largest exponent. Few large parts make
// it long and many make the chain's sum over them long; short_parts balances the two (12 of 64 x 768: 6 us, latency).
template <int M, int kSource>
__device__ __forceinline__ void gram(const Matrices& m, const MomentumScalars& s) {
    constexpr int B = M / 32, kMine = (B * B + 3) / 4, LD = kStep + 8, kPart = M * LD;
    constexpr bool kLow = kSource != 0;                  // bf16 values are exact in one part
    __shared__ __align__(16) f16 lds[(kLow ? 2 : 1) * kPart];
    __shared__ float most[4];
    if (skipped(s.clip)) return;
    const float clip = s.clip != nullptr ? *s.clip : 1.0f;
    uint32_t part;
    const Desc d = find(m, kByPart, blockIdx.x, &part);
    const bool tall = d.rows > d.cols;
    const int32_t n = tall ? d.rows : d.cols, steps = (n + kStep - 1) / kStep;
    const int32_t from = static_cast<int32_t>(static_cast<int64_t>(steps) * part / d.parts);
    const int32_t to = static_cast<int32_t>(static_cast<int64_t>(steps) * (part + 1) / d.parts);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    f32x16 acc[kMine] = {};
    int e = kEmpty;
    for (int32_t st = from; st < to; ++st) {
        Held<M> h = {};
        hold<M, kSource, true>(d, tall, st * kStep, s, clip, h);
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < Held<M>::kBlocks; ++i)
#pragma unroll
            for (int k = 0; k < 16; ++k) big = fmaxf(big, fabsf(h.v[i][k / 4][k % 4]));
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
        if (lane == 0) most[wave] = big;
        __syncthreads();                                 // and the step before has been multiplied
        big = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        const int here = big == 0.0f ? kEmpty : isfinite(big) ? ilogbf(big) : 127;
        if (here > e) {
            const float shrink = ldexpf(1.0f, 2 * (e - here));
#pragma unroll
            for (int i = 0; i < kMine; ++i) acc[i] *= shrink;
            e = here;
        }
        split<M, false, kLow>(h, tall, 13 - e, LD, lds, kPart);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int b = wave + 4 * i;
            if (B * B % 4 != 0 && b >= B * B) break;
            const f16* const x = lds + (b / B * 32 + lane % 32) * LD + lane / 32 * 8;
            const f16* const y = lds + (b % B * 32 + lane % 32) * LD + lane / 32 * 8;
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk) {
                const f16x8 xh = *reinterpret_cast<const f16x8*>(x + kk * 16), yh = *reinterpret_cast<const f16x8*>(y + kk * 16);
                acc[i] = mfma(xh, yh, acc[i]);
                if constexpr (kLow) {
                    const f16x8 xl = *reinterpret_cast<const f16x8*>(x + kPart + kk * 16),
                                yl = *reinterpret_cast<const f16x8*>(y + kPart + kk * 16);
                    acc[i] = mfma(xl, yh, mfma(xh, yl, acc[i]));
                }
            }
        }
    }
    float* const out = reinterpret_cast<float*>(m.ws + d.short_ws + short_area_bytes(M, part));
    if (threadIdx.x == 0) m.part_exponent[d.first[kByPart] + static_cast<int32_t>(part)] = e;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int b = wave + 4 * i;
        if (B * B % 4 != 0 && b >= B * B) break;
        *reinterpret_cast<f32x16*>(out + (b * 64 + lane) * 16) = acc[i];
    }
}

// A wave's 32 x 32 blocks of an M x M matrix: one, or with M = 128, where a wave for each would read LDS too often, two side
// by side.
template <int M>
struct ChainShape {
    static constexpr int kBlocks = M == 128 ? 2 : 1, kAcross = M / 32 / kBlocks, kWaves = M / 32 * kAcross;
};

// All steps of one matrix, on A. One compute unit a matrix, so bound by the latency of products that wait for one another,
// four a step of three MFMAs each and LDS reads between: five steps take 22 us at 64 x 64, 38 at 96, 78 at 128, for one
// matrix or 256.
template <int M>
__device__ __forceinline__ void chain(const Matrices& m, const ShortProgram& program, double eps, const float* clip) {
    constexpr int NB = ChainShape<M>::kBlocks, kWaves = ChainShape<M>::kWaves, LD = M + 8, kPart = M * LD, kSlot = 2 * kPart;
    constexpr bool kGlobalQ = M == 128;                  // three matrices of two parts do not fit the LDS
    __shared__ __align__(16) f16 lds[(kGlobalQ ? 2 : 3) * kSlot];
    __shared__ double traces[kWaves];
    if (skipped(clip)) return;
    const Desc d = matrix(m, blockIdx.x);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int bi = wave / ChainShape<M>::kAcross, bj = wave % ChainShape<M>::kAcross * NB;      // blocks bi, bj + n
    struct Blocks {
        f32x16 v[NB];
    };
    int e = kEmpty;
    for (int p = 0; p < d.parts; ++p) e = max(e, m.part_exponent[d.first[kByPart] + p]);
    Blocks a = {};
    const float* parts = reinterpret_cast<const float*>(m.ws + d.short_ws + short_area_bytes(M, 0));
    parts += ((bi * (M / 32) + bj) * 64 + lane) * 16;
#pragma unroll 4
    for (int p = 0; p < d.parts; ++p, parts += M * M) {
        const float scale = ldexpf(1.0f, 2 * (m.part_exponent[d.first[kByPart] + p] - e));
#pragma unroll
        for (int n = 0; n < NB; ++n) a.v[n] += *reinterpret_cast<const f32x16*>(parts + n * 1024) * scale;
    }
    double trace = 0.0;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (bi == bj + n && block_row(k) == lane % 32) trace += a.v[n][k];
    trace = ::zero::dev::wave_sum(trace);
    if (lane == 0) traces[wave] = trace;
    __syncthreads();
    trace = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) trace += traces[w];
    // |u| = sqrt(trace) 2^(e - 13)
    double factor = 0.0;
    if (isfinite(trace) && trace > 0.0) {
        const double unit = ldexp(1.0, e - 13);
        factor = unit / (sqrt(trace) * unit + eps);
    } else if (trace != 0.0) {
        factor = __builtin_nan("");
    }
    if (threadIdx.x == 0) m.short_scale[d.id] = ShortScale{trace == 0.0 ? 0 : e, static_cast<float>(factor)};
    const float unit_a = static_cast<float>(factor * factor * program.first);
#pragma unroll
    for (int n = 0; n < NB; ++n) a.v[n] *= unit_a;

    f16* const final_q = reinterpret_cast<f16*>(m.ws + d.short_ws);
    // times() takes its right factor's columns, so a matrix is stored by rows as a left factor and by columns as a right
    // one. All are symmetric but for roundings, but with A' = C A C^T and Q' = C Q in this order the roundings of C cancel
    // (A' stays the A of Q' X); with A C C they grow by a^2 a step (1e-3 of the result against 3e-5).
    // A lane holds a row's values where the factors are swapped in the MFMA, a column's where not: it writes four at once.
    constexpr std::true_type kByRows{};
    constexpr std::false_type kByColumns{};
    // The lane's values: with turned those of row (or column) 32 (bj + n) + lane % 32 from place 32 bi on, else the other way.
    auto put = [&](bool turned, const Blocks& x, f16* to, int ld, int part) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            f16* const at = to + ((turned ? bj + n : bi) * 32 + lane % 32) * ld + (turned ? bi : bj + n) * 32 + lane / 32 * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f16x4 hi, lo;
                split4(x.v[n][q * 4], x.v[n][q * 4 + 1], x.v[n][q * 4 + 2], x.v[n][q * 4 + 3], &hi, &lo);
                *reinterpret_cast<f16x4*>(at + q * 8) = hi;
                *reinterpret_cast<f16x4*>(at + q * 8 + part) = lo;
            }
        }
    };
    // The blocks bi, bj + n (turned: bj + n, bi) of x y, from the rows of x and the columns of y.
    auto times = [&](auto by_rows, bool turned, const f16* x, const f16* y, int y_ld, int y_part, float scale) {
        Blocks sum = {};
#pragma unroll
        for (int kk = 0; kk < M / 16; ++kk) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const f16* const xr = x + ((turned ? bj + n : bi) * 32 + lane % 32) * LD + lane / 32 * 8 + kk * 16;
                const f16* const yr = y + ((turned ? bi : bj + n) * 32 + lane % 32) * y_ld + lane / 32 * 8 + kk * 16;
                const f16x8 xh = *reinterpret_cast<const f16x8*>(xr), xl = *reinterpret_cast<const f16x8*>(xr + kPart);
                const f16x8 yh = *reinterpret_cast<const f16x8*>(yr), yl = *reinterpret_cast<const f16x8*>(yr + y_part);
                f32x16& s = sum.v[n];
                s = by_rows ? mfma(yl, xh, s) : mfma(xh, yl, s);
                s = by_rows ? mfma(yh, xl, s) : mfma(xl, yh, s);
                s = by_rows ? mfma(yh, xh, s) : mfma(xh, yh, s);
            }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) sum.v[n] *= scale;
        return sum;
    };
    f16* const slot_a = lds;
    f16* const slot_c = lds + kSlot;
    constexpr int kQLd = kGlobalQ ? M : LD, kQPart = kGlobalQ ? M * M : kPart;
    // Q: in LDS, or the matrix of this step and of the next in turn.
    auto slot_q = [&](int step) { return kGlobalQ ? final_q + (1 + step % 2) * 2 * M * M : lds + 2 * kSlot; };
    put(true, a, slot_a, LD, kPart);
    for (int32_t i = 0; i < program.n_steps; ++i) {
        const ShortStep& s = program.step[i];
        const bool last = i + 1 == program.n_steps;
        __syncthreads();
        // Turned blocks by rows: A is symmetric, so the lane's values of A, of a column, are those of the row it needs.
        Blocks c = times(kByRows, true, slot_a, slot_a, LD, kPart, s.c);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                c.v[n][k] += s.b * a.v[n][k];
                if (bi == bj + n && block_row(k) == lane % 32) c.v[n][k] += s.a;
            }
        put(true, c, slot_c, LD, kPart);
        if (i == 0 && last) put(true, c, final_q, M, M * M);
        __syncthreads();
        Blocks t = {}, q = {};
        if (last) {
            if (i > 0) q = times(kByRows, false, slot_c, slot_q(i - 1), kQLd, kQPart, s.q);
        } else {
            t = times(kByRows, false, slot_c, slot_a, LD, kPart, s.t);
            if (i > 0) q = times(kByColumns, false, slot_c, slot_q(i - 1), kQLd, kQPart, s.q);
        }
        __syncthreads();
        if (last) {
            if (i > 0) put(false, q, final_q, M, M * M);
            break;
        }
        if (i > 0) put(true, q, slot_q(i), kQLd, kQPart);
        if (i == 0) {                                    // Q = C, by columns
            for (int at = threadIdx.x; at < 2 * M * M / 4; at += kWaves * 64) {
                const int r = at / (M * M / 4), c4 = at / M % (M / 4) * 4, column = at % M;
                const f16* const from = slot_c + r * kPart + c4 * LD + column;
                *reinterpret_cast<f16x4*>(slot_q(0) + r * kQPart + column * kQLd + c4) =
                    f16x4{from[0], from[LD], from[2 * LD], from[3 * LD]};
            }
        }
        put(false, t, slot_a, LD, kPart);
        __syncthreads();
        a = times(kByColumns, false, slot_a, slot_c, LD, kPart, s.next);
        __syncthreads();
        put(true, a, slot_a, LD, kPart);
    }
}

// Q X of a part, and the last step with it.
template <int M, int kSource, int kEnd>
__device__ __forceinline__ void apply(const Matrices& m, const MomentumScalars& s, const Update& u, float last) {
    constexpr int B = M / 32, kMine = (2 * B + 3) / 4, LD = M + 8, kPart = kStep * LD, kWideLd = kStep + 8;
    constexpr bool kLow = kSource != 0;
    constexpr int kOut = M * kWideLd > kStep * LD ? M * kWideLd : kStep * LD;
    __shared__ __align__(16) f16 lds[(kLow ? 2 : 1) * kPart];
    __shared__ __align__(16) f16 out[kOut];
    if (skipped(s.clip)) return;
    const float clip = s.clip != nullptr ? *s.clip : 1.0f;
    uint32_t part;
    const Desc d = find(m, kByPart, blockIdx.x, &part);
    const bool tall = d.rows > d.cols;
    const int32_t n = tall ? d.rows : d.cols, steps = (n + kStep - 1) / kStep;
    const int32_t from = static_cast<int32_t>(static_cast<int64_t>(steps) * part / d.parts);
    const int32_t to = static_cast<int32_t>(static_cast<int64_t>(steps) * (part + 1) / d.parts);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const ShortScale scale = m.short_scale[d.id];
    const float alpha = scale.factor * last, rate = static_cast<float>(u.lr * d.scale);
    // A wave's blocks: rows of Q b % B, columns of the step b / B.
    const f16* const q = reinterpret_cast<const f16*>(m.ws + d.short_ws);
    f16x8 qh[kMine][M / 16], ql[kMine][M / 16];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const f16* const at = q + ((wave + 4 * i) % B * 32 + lane % 32) * M + lane / 32 * 8;
#pragma unroll
        for (int kk = 0; kk < M / 16; ++kk) {
            qh[i][kk] = *reinterpret_cast<const f16x8*>(at + kk * 16);
            ql[i][kk] = *reinterpret_cast<const f16x8*>(at + M * M + kk * 16);
        }
    }
    for (int32_t st = from; st < to; ++st) {
        Held<M> h = {};
        hold<M, kSource, false>(d, tall, st * kStep, s, clip, h);
        split<M, true, kLow>(h, tall, 13 - scale.exponent, LD, lds, kPart);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int b = wave + 4 * i, row = b % B * 32, col = b / B * 32;
            if (2 * B % 4 != 0 && b >= 2 * B) break;
            const f16* const x = lds + (col + lane % 32) * LD + lane / 32 * 8;
            f32x16 acc = {};
#pragma unroll
            for (int kk = 0; kk < M / 16; ++kk) {
                const f16x8 xh = *reinterpret_cast<const f16x8*>(x + kk * 16);
                acc = mfma(qh[i][kk], xh, mfma(ql[i][kk], xh, acc));
                if constexpr (kLow) acc = mfma(qh[i][kk], *reinterpret_cast<const f16x8*>(x + kPart + kk * 16), acc);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
                const u32x2_t bits = {::zero::dev::pack_bf16(alpha * acc[g * 4], alpha * acc[g * 4 + 1]),
                                      ::zero::dev::pack_bf16(alpha * acc[g * 4 + 2], alpha * acc[g * 4 + 3])};
                const f16x4 v = __builtin_bit_cast(f16x4, bits);
                const int r = row + g * 8 + lane / 32 * 4, c = col + lane % 32;
                if (tall)
                    *reinterpret_cast<f16x4*>(out + c * LD + r) = v;
                else
                    *reinterpret_cast<f16x4*>(out + (r + lane % 4) * kWideLd + c - lane % 4) = quad_transpose(v);
            }
        }
        __syncthreads();
        const int32_t r0 = tall ? st * kStep : 0, c0 = tall ? 0 : st * kStep;
        const int out_rows = tall ? kStep : M, pieces = (tall ? M : kStep) / 8, ld = tall ? LD : kWideLd;
        for (int at = threadIdx.x; at < out_rows * pieces; at += kThreads) {
            const int r = at / pieces, piece = at % pieces;
            const int32_t c = c0 + piece * 8;
            int here = r0 + r < d.rows ? d.cols - c : 0;
            here = here < 0 ? 0 : here > 8 ? 8 : here;
            const int64_t first = static_cast<int64_t>(r0 + r) * d.cols + c;
            float w[8];
            if constexpr (kEnd == 2) {
                read4(d.master, first, here < 4 ? here : 4, w);
                read4(d.master, first + 4, here < 4 ? 0 : here - 4, w + 4);
            }
            const f16x8 o = *reinterpret_cast<const f16x8*>(out + r * ld + piece * 8);
            uint16_t bits[8];
            __builtin_memcpy(bits, &o, sizeof(bits));
            finish8<kEnd>(d, u, rate, first, here, bits, w);
        }
    }
}

template <int M, int kSource>
__global__ __launch_bounds__(kThreads) void short_gram_kernel(Matrices m, MomentumScalars s) {
    gram<M, kSource>(m, s);
}

template <int M>
__global__ __launch_bounds__(64 * ChainShape<M>::kWaves) void short_chain_kernel(Matrices m, ShortProgram program, double eps,
                                                                            const float* clip) {
    chain<M>(m, program, eps, clip);
}

template <int M, int kSource, int kEnd>
__global__ __launch_bounds__(kThreads) void short_apply_kernel(Matrices m, MomentumScalars s, Update u, float last) {
    apply<M, kSource, kEnd>(m, s, u, last);
}

template <int M, int kSource>
zero_status launch(const Matrices& m, const MomentumScalars& s, const Update& u,
                   const ShortProgram& program, double eps, hipStream_t stream, const char* who) {
    const dim3 parts(m.total[kByPart]);
    hipLaunchKernelGGL((short_gram_kernel<M, kSource>), parts, dim3(kThreads), 0, stream, m, s);
    zero_status st = zero::check_hip(hipGetLastError(), who);
    if (st != ZERO_OK) return st;
    hipLaunchKernelGGL((short_chain_kernel<M>), dim3(m.matrices), dim3(64 * ChainShape<M>::kWaves), 0, stream, m, program, eps, s.clip);
    st = zero::check_hip(hipGetLastError(), who);
    if (st != ZERO_OK) return st;
    hipLaunchKernelGGL((short_apply_kernel<M, kSource, kSource == 2 ? 2 : 1>), parts, dim3(kThreads), 0, stream, m, s, u,
                       program.last);
    return zero::check_hip(hipGetLastError(), who);
}

template <int M>
zero_status launch(int source, const Matrices& m, const MomentumScalars& s, const Update& u,
                   const ShortProgram& program, double eps, hipStream_t stream, const char* who) {
    if (source == 0) return launch<M, 0>(m, s, u, program, eps, stream, who);
    if (source == 1) return launch<M, 1>(m, s, u, program, eps, stream, who);
    return launch<M, 2>(m, s, u, program, eps, stream, who);
}

}  // namespace

namespace zero {
namespace muon {

zero_status launch_short(int source, const dev::Matrices& m, const dev::MomentumScalars& s,
                         const dev::Update& u, const ShortProgram& program, double eps, hipStream_t stream, const char* who) {
    if (m.side == 64) return launch<64>(source, m, s, u, program, eps, stream, who);
    if (m.side == 96) return launch<96>(source, m, s, u, program, eps, stream, who);
    return launch<128>(source, m, s, u, program, eps, stream, who);
}

}  // namespace muon
}  // namespace zero
