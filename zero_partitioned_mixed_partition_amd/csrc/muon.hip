// Muon on gfx950: matrices orthogonalised by Newton-Schulz steps, and the
// update of weight matrices by their orthogonalised momentum. The products
// that one call runs, and the layout of its workspace, are muon_plan.hpp's.
//
// "Zero Redundancy Optimizer (ZeRO) and Fully Sharded Data Parallelism (FSDP):
// Mathematical Foundations ...", section "Execution Flow for ZeRO-1", steps 3-4
// (the rank updates its own fp32 master weights and emits 16-bit parameters),
// with Muon's update in AdamW's place.
//
// One call is: the momentum pass (momentum written, |u|^2 as fixed-order
// partial sums), the packing (u scaled by a power of two into fp16, in both
// orders of storage and padded to whole tiles, so that every product reads
// rows of contiguous K and needs no bounds checks), then the products, each one
// launch over the tiles of every matrix of the call; the last one's epilogue is
// the weight update.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "device_common.hpp"
#include "internal.hpp"
#include "muon_plan.hpp"
#include "pieces.hpp"

#pragma clang fp contract(off)

namespace {

using zero::muon::Desc;
using zero::muon::Kind;
using zero::muon::Product;

typedef _Float16 f16;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTile = 128;        // a workgroup's tile of a product, and the padding's unit
constexpr int kDepth = 64;        // K elements of one LDS stage

// The matrices of one call: a device table of descriptors, or (table NULL) a stack of equal matrices described by its
// first.
struct Matrices {
    const Desc* table;
    const uint32_t* index[3];     // per grid, the descriptor of each workgroup
    Desc base;
    int64_t src_bytes;            // from one matrix of a stack to the next
    int64_t numel;
    int64_t area;
    uint32_t per[3];              // workgroups of one matrix of a stack, per grid
    uint32_t total[3];
    double* partials;
    float* kappa;
    char* ws;
};

// The matrix of workgroup t of a grid, and the workgroup's number within it.
__device__ __forceinline__ Desc find(const Matrices& m, int grid, uint32_t t, uint32_t* local) {
    if (m.table != nullptr) {
        const Desc d = m.table[m.index[grid][t]];
        *local = t - static_cast<uint32_t>(d.first[grid]);
        return d;
    }
    const uint32_t i = t / m.per[grid];
    *local = t - i * m.per[grid];
    Desc d = m.base;
    const int64_t at = m.numel * i;
    d.src = static_cast<const char*>(d.src) + m.src_bytes * i;
    if (d.momentum != nullptr) d.momentum += at;
    if (d.master != nullptr) d.master += at;
    d.out += at;
    d.ws += m.area * i;
    d.first_partial = d.chunks * static_cast<int32_t>(i);
    d.id = static_cast<int32_t>(i);
    return d;
}

// What the momentum pass computes per element.
struct MomentumScalars {
    float mu;
    int32_t nesterov;
    const float* clip;            // NULL: 1
};

__device__ __forceinline__ bool skipped(const float* clip) { return clip != nullptr && !isfinite(*clip); }

__device__ __forceinline__ float gradient(const Desc& d, int64_t i, float clip) {
    return zero::dev::bf16_to_f32(static_cast<const uint16_t*>(d.src)[i]) * clip;
}

// The matrix to orthogonalise at element i. kSource: 0 bf16, 1 fp32, 2 momentum (already updated) and gradient.
template <int kSource>
__device__ __forceinline__ float input(const Desc& d, int64_t i, const MomentumScalars& s, float clip) {
    if constexpr (kSource == 0) return zero::dev::bf16_to_f32(static_cast<const uint16_t*>(d.src)[i]);
    if constexpr (kSource == 1) return static_cast<const float*>(d.src)[i];
    const float buf = d.momentum[i];
    return s.nesterov ? gradient(d, i, clip) + s.mu * buf : buf;
}

// Momentum and squared norm: each workgroup takes one chunk of one matrix.
template <int kSource>
__global__ __launch_bounds__(kThreads) void momentum_kernel(Matrices m, MomentumScalars s) {
    __shared__ double lds[kThreads / zero::dev::kWave];
    if (skipped(s.clip)) return;
    const float clip = s.clip != nullptr ? *s.clip : 1.0f;
    uint32_t c;
    const Desc d = find(m, zero::muon::kByChunk, blockIdx.x, &c);
    const int64_t n = static_cast<int64_t>(d.rows) * d.cols;
    const int64_t lo = d.chunk * c, hi = lo + d.chunk < n ? lo + d.chunk : n;
    double sum = 0.0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        if constexpr (kSource == 2) d.momentum[i] = s.mu * d.momentum[i] + gradient(d, i, clip);
        const double u = input<kSource>(d, i, s, clip);
        sum += u * u;
    }
    sum = zero::dev::block_sum<kThreads>(sum, lds);
    if (threadIdx.x == 0) m.partials[d.first_partial + static_cast<int64_t>(c)] = sum;
}

__device__ __forceinline__ f16* buffer(const Matrices& m, const Desc& d, int32_t which) {
    const int64_t mn = static_cast<int64_t>(d.M) * d.N, mm = static_cast<int64_t>(d.M) * d.M;
    f16* const at = reinterpret_cast<f16*>(m.ws + d.ws);
    switch (which) {
        case zero::muon::kX: return at;
        case zero::muon::kT0: return at + mn;
        case zero::muon::kT1: return at + 2 * mn;
        case zero::muon::kS0: return at + 3 * mn;
        case zero::muon::kS1: return at + 3 * mn + mm;
        case zero::muon::kS2: return at + 3 * mn + 2 * mm;
        default: return at + 3 * mn + 3 * mm;
    }
}

// Packs a 128 x 128 tile of the padded matrix: u * 2^(13 - e), where |u| lies in [2^e, 2^(e + 1)), as fp16 in both
// orders, and with kLowPart what the rounding left. X is 2^-14 kappa times what is held.
template <int kSource, bool kLowPart>
__global__ __launch_bounds__(kThreads) void pack_kernel(Matrices m, MomentumScalars s, double eps) {
    constexpr int kStride = kTile + 2;
    __shared__ f16 tile[kTile * kStride];
    __shared__ double lds[kThreads / zero::dev::kWave];
    __shared__ double total;
    if (skipped(s.clip)) return;
    const float clip = s.clip != nullptr ? *s.clip : 1.0f;
    uint32_t t;
    const Desc d = find(m, zero::muon::kByTile, blockIdx.x, &t);
    double sum = 0.0;
    for (int32_t i = threadIdx.x; i < d.chunks; i += kThreads) sum += m.partials[d.first_partial + i];
    sum = zero::dev::block_sum<kThreads>(sum, lds);
    if (threadIdx.x == 0) total = sum;
    __syncthreads();
    const double norm = sqrt(total);
    int e = 0;
    float kappa = 0.0f;
    if (isfinite(norm) && norm > 0.0) {
        e = ilogb(norm);
        kappa = static_cast<float>(ldexp(1.0, e + 1) / (norm + eps));
    } else if (norm != 0.0) {
        kappa = __builtin_nanf("");
    }
    if (t == 0 && threadIdx.x == 0) m.kappa[d.id] = kappa;

    // The source's rows run along `tall ? N : M`.
    const bool tall = d.rows > d.cols;
    const int32_t padded_rows = tall ? d.N : d.M, padded_cols = tall ? d.M : d.N;
    const uint32_t tiles = padded_cols / kTile;
    const int32_t r0 = static_cast<int32_t>(t / tiles) * kTile, c0 = static_cast<int32_t>(t % tiles) * kTile;
    f16* const along = buffer(m, d, tall ? zero::muon::kT0 : zero::muon::kX);
    f16* const across = buffer(m, d, tall ? zero::muon::kX : zero::muon::kT0);
    f16* const low = buffer(m, d, zero::muon::kLow);
    constexpr int kPer = kTile * kTile / kThreads;
    f16 rest[kLowPart ? kPer : 1];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = threadIdx.x + k * kThreads, r = at / kTile, c = at % kTile;
        float x = 0.0f;
        if (r0 + r < d.rows && c0 + c < d.cols)
            x = ldexpf(input<kSource>(d, static_cast<int64_t>(r0 + r) * d.cols + c0 + c, s, clip), 13 - e);
        const f16 h = static_cast<f16>(x);
        if constexpr (kLowPart) rest[k] = static_cast<f16>(x - static_cast<float>(h));
        tile[r * kStride + c] = h;
        along[static_cast<int64_t>(r0 + r) * padded_cols + c0 + c] = h;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = threadIdx.x + k * kThreads, c = at / kTile, r = at % kTile;
        across[static_cast<int64_t>(c0 + c) * padded_rows + r0 + r] = tile[r * kStride + c];
    }
    if constexpr (kLowPart) {      // [N][M], as kT0
        if (tall) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int at = threadIdx.x + k * kThreads, r = at / kTile, c = at % kTile;
                low[static_cast<int64_t>(r0 + r) * padded_cols + c0 + c] = rest[k];
            }
            return;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int at = threadIdx.x + k * kThreads;
            tile[at / kTile * kStride + at % kTile] = rest[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int at = threadIdx.x + k * kThreads, c = at / kTile, r = at % kTile;
            low[static_cast<int64_t>(c0 + c) * padded_rows + r0 + r] = tile[r * kStride + c];
        }
    }
}

// The weight update of the last product's epilogue.
struct Update {
    double lr;
    float decay;                  // 1 - lr * weight_decay
    const float* clip;
};

// An operand's tile rows in LDS: kDepth values, eight 16-byte pieces a row, piece p of row r at place p ^ (r / 2 % 8),
// so that 16 rows' pieces of one column lie in all banks.
__device__ __forceinline__ int lds_place(int r, int p) { return r * kDepth + ((p ^ ((r >> 1) & 7)) << 3); }

// One 128 x 128 tile of a product: four waves of 64 x 64, each 2 x 2 MFMA tiles of 32 x 32.
template <bool kSquareOut, int kEnd>     // kEnd: 0 workspace, 1 orthogonalised matrix, 2 weight update
__global__ __launch_bounds__(kThreads) void product_kernel(Matrices m, Product p, Update u) {
    __shared__ f16 lds[2 * kTile * kDepth];
    if (kEnd == 2 && skipped(u.clip)) return;
    uint32_t t;
    const Desc d = find(m, kSquareOut ? zero::muon::kByPair : zero::muon::kByTile, blockIdx.x, &t);
    const bool tall = d.rows > d.cols;
    int32_t bi, bj;
    if constexpr (kSquareOut) {           // tile t of the lower triangle, row by row
        bi = static_cast<int32_t>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
        while (static_cast<uint32_t>(bi) * (bi + 1) / 2 > t) --bi;
        while (static_cast<uint32_t>(bi + 1) * (bi + 2) / 2 <= t) ++bi;
        bj = static_cast<int32_t>(t - static_cast<uint32_t>(bi) * (bi + 1) / 2);
    } else {
        const uint32_t tiles = (tall ? d.M : d.N) / kTile;
        bi = static_cast<int32_t>(t / tiles);
        bj = static_cast<int32_t>(t % tiles);
    }
    const int32_t K = p.kind == Kind::kGram ? d.N : d.M;
    const f16* left = buffer(m, d, p.lhs);
    const f16* right = buffer(m, d, p.rhs);
    const f16* const low = buffer(m, d, zero::muon::kLow);
    if (!kSquareOut && tall) {            // rows of the output are the source's: X^T on the left
        const f16* const x = left;
        left = right;
        right = x;
    }

    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int wr = wave / 2 * 64, wc = wave % 2 * 64;
    f32x16 acc[2][2] = {};
    const int passes = p.with_low ? 2 : 1;
    for (int pass = 0; pass < passes; ++pass) {
        const f16* a = left;
        const f16* b = right;
        if (pass == 1) (tall ? a : b) = low;
        a += static_cast<int64_t>(bi) * kTile * K;
        b += static_cast<int64_t>(bj) * kTile * K;
        for (int32_t k0 = 0; k0 < K; k0 += kDepth) {
            f16x8 ra[4], rb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = threadIdx.x + i * kThreads, r = at / 8, c = at % 8;
                ra[i] = *reinterpret_cast<const f16x8*>(a + static_cast<int64_t>(r) * K + k0 + c * 8);
                rb[i] = *reinterpret_cast<const f16x8*>(b + static_cast<int64_t>(r) * K + k0 + c * 8);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = threadIdx.x + i * kThreads, r = at / 8, c = at % 8;
                *reinterpret_cast<f16x8*>(lds + lds_place(r, c)) = ra[i];
                *reinterpret_cast<f16x8*>(lds + kTile * kDepth + lds_place(r, c)) = rb[i];
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kDepth / 16; ++kk) {
                f16x8 fa[2], fb[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = kk * 2 + lane / 32;
                    fa[i] = *reinterpret_cast<const f16x8*>(lds + lds_place(wr + i * 32 + lane % 32, c));
                    fb[i] = *reinterpret_cast<const f16x8*>(lds + kTile * kDepth + lds_place(wc + i * 32 + lane % 32, c));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }
    }

    // A lane holds one column of each MFMA tile, four consecutive rows at a time.
    float alpha = p.alpha;
    if (p.kappa_power > 0) {
        const float kappa = m.kappa[d.id];
        alpha = p.kappa_power == 2 ? alpha * (kappa * kappa) : alpha * kappa;
    }
    const int32_t row0 = bi * kTile + wr + lane / 32 * 4, col0 = bj * kTile + wc + lane % 32;
    if constexpr (kSquareOut) {
        const f16* const add = p.add != zero::muon::kNone ? buffer(m, d, p.add) : nullptr;
        f16* const out = buffer(m, d, p.out);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int32_t r = row0 + i * 32 + q * 8, c = col0 + j * 32;
                    const int64_t mirrored = static_cast<int64_t>(c) * d.M + r;
                    f16x4 old = {};
                    if (add != nullptr) old = *reinterpret_cast<const f16x4*>(add + mirrored);
                    f16x4 v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = alpha * acc[i][j][q * 4 + k] + p.beta * static_cast<float>(old[k]);
                        if (r + k == c) x += p.diag;
                        v[k] = static_cast<f16>(x);
                        if (bi != bj) out[static_cast<int64_t>(r + k) * d.M + c] = v[k];
                    }
                    *reinterpret_cast<f16x4*>(out + mirrored) = v;
                }
    } else {
        const int32_t out_rows = tall ? d.N : d.M, out_cols = tall ? d.M : d.N;
        f16* const along = kEnd == 0 ? buffer(m, d, tall ? p.out_t : p.out) : nullptr;
        f16* const across = kEnd == 0 ? buffer(m, d, tall ? p.out : p.out_t) : nullptr;
        const float rate = static_cast<float>(u.lr * d.scale);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int32_t r = row0 + i * 32 + q * 8, c = col0 + j * 32;
                    f16x4 v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x = alpha * acc[i][j][q * 4 + k];
                        if constexpr (kEnd == 0) {
                            v[k] = static_cast<f16>(x);
                            along[static_cast<int64_t>(r + k) * out_cols + c] = v[k];
                        } else if (r + k < d.rows && c < d.cols) {
                            const int64_t at = static_cast<int64_t>(r + k) * d.cols + c;
                            const uint32_t o = zero::dev::f32_to_bf16(x);
                            if constexpr (kEnd == 1) {
                                d.out[at] = static_cast<uint16_t>(o);
                            } else {
                                float w = d.master[at] * u.decay;
                                w = w - rate * zero::dev::bf16_to_f32(o);
                                d.master[at] = w;
                                d.out[at] = static_cast<uint16_t>(zero::dev::f32_to_bf16(w));
                            }
                        }
                    }
                    if constexpr (kEnd == 0)
                        *reinterpret_cast<f16x4*>(across + static_cast<int64_t>(c) * out_rows + r) = v;
                }
    }
}

// ------------------------------------------------------------ launches

// One call's arguments besides its matrices.
struct Call {
    const double* coefficients;
    int32_t n_steps;
    double eps;
    int source;                   // 0 bf16, 1 fp32, 2 momentum and gradient
    MomentumScalars momentum;
    Update update;
    double cost[2];               // of one pair and single steps, and of pairs
};

template <int kSource, int kEnd>
zero_status launch_all(const Matrices& m, const Call& c, const std::vector<Product>& program, hipStream_t stream,
                       const char* who) {
    hipLaunchKernelGGL(momentum_kernel<kSource>, dim3(m.total[zero::muon::kByChunk]), dim3(kThreads), 0, stream, m,
                       c.momentum);
    zero_status st = zero::check_hip(hipGetLastError(), who);
    if (st != ZERO_OK) return st;
    const dim3 tiles(m.total[zero::muon::kByTile]), pairs(m.total[zero::muon::kByPair]);
    hipLaunchKernelGGL((pack_kernel<kSource, kSource != 0>), tiles, dim3(kThreads), 0, stream, m, c.momentum, c.eps);
    st = zero::check_hip(hipGetLastError(), who);
    for (const Product& p : program) {
        if (st != ZERO_OK) return st;
        if (p.kind == Kind::kGram || p.kind == Kind::kSquare)
            hipLaunchKernelGGL((product_kernel<true, 0>), pairs, dim3(kThreads), 0, stream, m, p, c.update);
        else if (p.kind == Kind::kApply)
            hipLaunchKernelGGL((product_kernel<false, 0>), tiles, dim3(kThreads), 0, stream, m, p, c.update);
        else
            hipLaunchKernelGGL((product_kernel<false, kEnd>), tiles, dim3(kThreads), 0, stream, m, p, c.update);
        st = zero::check_hip(hipGetLastError(), who);
    }
    return st;
}

zero_status launch(const Matrices& m, const Call& c, hipStream_t stream, const char* who) {
    std::vector<Product> program;
    // Pairs where they save a twentieth of the multiplications or more: at equal cost the single steps, whose A comes
    // from X itself, are more exact (about 1.2e-3 of the result's norm against 1.5e-3 to 1.9e-3).
    const bool pairs = c.cost[1] < 0.95 * c.cost[0];
    try {
        const zero_status st = zero::muon::make_program(c.coefficients, c.n_steps, pairs, c.source != 0, &program, who);
        if (st != ZERO_OK) return st;
    } catch (const std::bad_alloc&) {
        return zero::fail(ZERO_ENOMEM, std::string(who) + ": host allocation failed");
    }
    if (c.source == 0) return launch_all<0, 1>(m, c, program, stream, who);
    if (c.source == 1) return launch_all<1, 1>(m, c, program, stream, who);
    return launch_all<2, 2>(m, c, program, stream, who);
}

zero_status check_workspace(const void* workspace, size_t bytes, int64_t need, const char* who) {
    const std::string w(who);
    if (!workspace) return zero::fail(ZERO_EINVAL, w + ": NULL workspace");
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return zero::fail(ZERO_EINVAL, w + ": workspace not 256-byte aligned");
    if (bytes < static_cast<size_t>(need))
        return zero::fail(ZERO_ENOSPACE, w + ": workspace holds " + std::to_string(bytes) + " bytes, " +
                                             std::to_string(need) + " needed");
    return ZERO_OK;
}

// ZERO_ERANGE for sides past the limits.
zero_status check_sides(int64_t rows, int64_t cols, const std::string& what) {
    if (std::min(rows, cols) > zero::muon::kMaxShort || std::max(rows, cols) > zero::muon::kMaxLong)
        return zero::fail(ZERO_ERANGE, what + ": " + std::to_string(rows) + " x " + std::to_string(cols) +
                                           " is past 65,536 on the shorter side or 2^22 on the longer");
    return ZERO_OK;
}

constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / kThreads - 1;      // fewer than 2^32 work-items a launch

// A stack's sizes: its first matrix's descriptor (sides, chunks), the workgroups and the workspace. ZERO_ERANGE where
// one launch does not hold it.
zero_status measure_stack(int64_t count, int64_t rows, int64_t cols, Matrices* m, int64_t* bytes, const char* who) {
    zero_status st = check_sides(rows, cols, who);
    if (st != ZERO_OK) return st;
    zero::muon::shape(&m->base, rows, cols, kTile);
    m->numel = rows * cols;
    m->area = zero::muon::area_bytes(m->base);
    for (int g = 0; g < 3; ++g) {
        const int64_t per = zero::muon::grid_count(m->base, g, kTile);
        if (count > kMaxBlocks / per)
            return zero::fail(ZERO_ERANGE, std::string(who) + ": more workgroups than one launch holds");
        m->per[g] = static_cast<uint32_t>(per);
        m->total[g] = static_cast<uint32_t>(per * count);
    }
    const int64_t head = zero::muon::head_bytes(count * m->base.chunks, count);
    if (count > (INT64_MAX - head) / m->area) return zero::fail(ZERO_ERANGE, std::string(who) + ": workspace overflows");
    *bytes = head + count * m->area;
    m->base.ws = head;
    return ZERO_OK;
}

void place(Matrices* m, void* workspace, int64_t partials) {
    m->ws = static_cast<char*>(workspace);
    m->partials = static_cast<double*>(workspace);
    m->kappa = reinterpret_cast<float*>(m->partials + partials);
}

// The counts of a stack. *empty: nothing to do.
zero_status check_counts(int64_t count, int64_t rows, int64_t cols, bool* empty, const char* who) {
    if (count < 0 || rows < 0 || cols < 0) return zero::fail(ZERO_EINVAL, std::string(who) + ": a count is negative");
    *empty = count == 0 || rows == 0 || cols == 0;
    return ZERO_OK;
}

zero_status check_eps(double eps, const char* who) {
    if (!(eps >= 0.0) || !std::isfinite(eps))
        return zero::fail(ZERO_EINVAL, std::string(who) + ": eps must be finite and not negative");
    return ZERO_OK;
}

zero_status muon_call(double lr, double momentum, int32_t nesterov, double weight_decay, const double* coefficients,
                      int32_t n_steps, double eps, const float* clip_scale, Call* c, const char* who) {
    const std::string w(who);
    if (!std::isfinite(lr) || lr < 0.0) return zero::fail(ZERO_EINVAL, w + ": lr must be finite and not negative");
    if (!(momentum >= 0.0 && momentum < 1.0)) return zero::fail(ZERO_EINVAL, w + ": momentum must lie in [0, 1)");
    if (!std::isfinite(weight_decay)) return zero::fail(ZERO_EINVAL, w + ": weight_decay is not finite");
    zero_status st = check_eps(eps, who);
    if (st == ZERO_OK) st = zero::muon::check_coefficients(coefficients, n_steps, who);
    if (st != ZERO_OK) return st;
    c->coefficients = coefficients;
    c->n_steps = n_steps;
    c->eps = eps;
    c->source = 2;
    c->momentum = MomentumScalars{static_cast<float>(momentum), nesterov != 0, clip_scale};
    c->update = Update{lr, static_cast<float>(1.0 - lr * weight_decay), clip_scale};
    return ZERO_OK;
}

// A call's cost with one pair and with pairs, summed over its matrices.
void add_cost(Call* c, const Desc& d) {
    for (int k = 0; k < 2; ++k) c->cost[k] += zero::muon::program_cost(c->n_steps, k != 0, d.M, d.N);
}

}  // namespace

extern "C" size_t zero_muon_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
    Matrices m{};
    int64_t bytes = 0;
    bool empty = false;
    if (check_counts(count, rows, cols, &empty, "zero_muon_workspace_bytes") != ZERO_OK || empty) return 0;
    if (measure_stack(count, rows, cols, &m, &bytes, "zero_muon_workspace_bytes") != ZERO_OK) return 0;
    return static_cast<size_t>(bytes);
}

extern "C" zero_status zero_orthogonalize(const void* x, int32_t x_type, uint16_t* out, int64_t count, int64_t rows,
                                          int64_t cols, const double* coefficients, int32_t n_steps, double eps,
                                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using zero::fail;
    static const char* const who = "zero_orthogonalize";
    zero::clear_error();
    if (x_type != ZERO_MATRIX_BF16 && x_type != ZERO_MATRIX_F32)
        return fail(ZERO_EINVAL, "zero_orthogonalize: x_type is neither ZERO_MATRIX_BF16 nor ZERO_MATRIX_F32");
    bool empty = false;
    zero_status st = check_counts(count, rows, cols, &empty, who);
    if (st == ZERO_OK) st = check_eps(eps, who);
    if (st == ZERO_OK) st = zero::muon::check_coefficients(coefficients, n_steps, who);
    if (st != ZERO_OK || empty) return st;
    if (!x || !out) return fail(ZERO_EINVAL, "zero_orthogonalize: NULL array");
    Matrices m{};
    int64_t need = 0;
    st = measure_stack(count, rows, cols, &m, &need, who);
    if (st == ZERO_OK) st = check_workspace(workspace, workspace_bytes, need, who);
    if (st != ZERO_OK) return st;
    const size_t n = static_cast<size_t>(count * m.numel), size = x_type == ZERO_MATRIX_F32 ? 4 : 2;
    const zero::Span wr[] = {{out, 2 * n, "out"}, {workspace, static_cast<size_t>(need), "workspace"}};
    const zero::Span rd[] = {{x, size * n, "x"}};
    const std::string clash = zero::first_overlap(wr, 2, rd, 1);
    if (!clash.empty()) return fail(ZERO_EINVAL, "zero_orthogonalize: " + clash);
    m.base.src = x;
    m.base.out = out;
    m.src_bytes = m.numel * static_cast<int64_t>(size);
    place(&m, workspace, count * m.base.chunks);
    Call c{};
    c.coefficients = coefficients;
    c.n_steps = n_steps;
    c.eps = eps;
    c.source = x_type == ZERO_MATRIX_F32 ? 1 : 0;
    add_cost(&c, m.base);
    return launch(m, c, stream, who);
}

extern "C" zero_status zero_muon_step(float* master, float* momentum, const uint16_t* grad, uint16_t* param_out,
                                      int64_t count, int64_t rows, int64_t cols, double lr, double mu,
                                      int32_t nesterov, double weight_decay, double scale,
                                      const double* coefficients, int32_t n_steps, double eps,
                                      const float* clip_scale, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    using zero::fail;
    static const char* const who = "zero_muon_step";
    zero::clear_error();
    bool empty = false;
    zero_status st = check_counts(count, rows, cols, &empty, who);
    Call c{};
    if (st == ZERO_OK)
        st = muon_call(lr, mu, nesterov, weight_decay, coefficients, n_steps, eps, clip_scale, &c, who);
    if (st == ZERO_OK && !std::isfinite(scale)) st = fail(ZERO_EINVAL, "zero_muon_step: scale is not finite");
    if (st != ZERO_OK || empty) return st;
    if (!master || !momentum || !grad || !param_out) return fail(ZERO_EINVAL, "zero_muon_step: NULL array");
    Matrices m{};
    int64_t need = 0;
    st = measure_stack(count, rows, cols, &m, &need, who);
    if (st == ZERO_OK) st = check_workspace(workspace, workspace_bytes, need, who);
    if (st != ZERO_OK) return st;
    const size_t n = static_cast<size_t>(count * m.numel);
    const zero::Span wr[] = {{master, 4 * n, "master"},
                             {momentum, 4 * n, "momentum"},
                             {param_out, 2 * n, "param_out"},
                             {workspace, static_cast<size_t>(need), "workspace"}};
    const zero::Span rd[] = {{grad, 2 * n, "grad"}};
    const std::string clash = zero::first_overlap(wr, 4, rd, 1);
    if (!clash.empty()) return fail(ZERO_EINVAL, "zero_muon_step: " + clash);
    m.base.src = grad;
    m.base.momentum = momentum;
    m.base.master = master;
    m.base.out = param_out;
    m.base.scale = scale;
    m.src_bytes = 2 * m.numel;
    place(&m, workspace, count * m.base.chunks);
    add_cost(&c, m.base);
    return launch(m, c, stream, who);
}

// ------------------------------------------------------------ a list of matrices

struct zero_muon_table {
    void* mem = nullptr;              // descriptors, then the three grids' indexes
    int device = -1;
    std::vector<Desc> descs;
    Matrices m{};
    int64_t partials = 0;
    int64_t bytes = 0;                // of the workspace
};

extern "C" void zero_muon_table_free(zero_muon_table* table) {
    if (!table) return;
    if (table->mem) (void)hipFree(table->mem);
    delete table;
}

namespace {

// Places the matrices in the workspace and the grids, and copies the descriptors and indexes to the device. Throws
// std::bad_alloc.
zero_status fill_table(zero_muon_table* tab, const char* who) {
    using zero::fail;
    const std::string w(who);
    if (tab->descs.empty()) return ZERO_OK;              // needs no device
    std::vector<uint32_t> index;
    size_t starts[3] = {};
    for (int g = 0; g < 3; ++g) {
        starts[g] = index.size();
        int64_t total = 0;
        for (size_t i = 0; i < tab->descs.size(); ++i) {
            Desc& d = tab->descs[i];
            const int64_t n = zero::muon::grid_count(d, g, kTile);
            if (n > kMaxBlocks - total) return fail(ZERO_ERANGE, w + ": more workgroups than one launch holds");
            d.first[g] = static_cast<int32_t>(total);
            index.insert(index.end(), static_cast<size_t>(n), static_cast<uint32_t>(i));
            total += n;
        }
        tab->m.total[g] = static_cast<uint32_t>(total);
    }
    for (size_t i = 0; i < tab->descs.size(); ++i) {
        Desc& d = tab->descs[i];
        d.id = static_cast<int32_t>(i);
        d.first_partial = static_cast<int32_t>(tab->partials);
        tab->partials += d.chunks;
    }
    tab->bytes = zero::muon::head_bytes(tab->partials, static_cast<int64_t>(tab->descs.size()));
    for (Desc& d : tab->descs) {
        d.ws = tab->bytes;
        const int64_t area = zero::muon::area_bytes(d);
        if (area > INT64_MAX - tab->bytes) return fail(ZERO_ERANGE, w + ": workspace overflows");
        tab->bytes += area;
    }
    zero_status st = zero::check_hip(hipGetDevice(&tab->device), "zero_muon_table_create: hipGetDevice");
    if (st != ZERO_OK) return st;
    const size_t table_bytes = tab->descs.size() * sizeof(Desc), index_bytes = index.size() * sizeof(uint32_t);
    st = zero::check_hip(hipMalloc(&tab->mem, table_bytes + index_bytes), "zero_muon_table_create: hipMalloc");
    if (st != ZERO_OK) return st;
    char* const at = static_cast<char*>(tab->mem);
    tab->m.table = reinterpret_cast<const Desc*>(at);
    for (int g = 0; g < 3; ++g) tab->m.index[g] = reinterpret_cast<const uint32_t*>(at + table_bytes) + starts[g];
    st = zero::check_hip(hipMemcpy(at, tab->descs.data(), table_bytes, hipMemcpyHostToDevice),
                         "zero_muon_table_create: hipMemcpy");
    if (st != ZERO_OK) return st;
    return zero::check_hip(hipMemcpy(at + table_bytes, index.data(), index_bytes, hipMemcpyHostToDevice),
                           "zero_muon_table_create: hipMemcpy");
}

}  // namespace

extern "C" zero_status zero_muon_table_create(float* const* masters, float* const* momenta,
                                              const uint16_t* const* grads, uint16_t* const* params_out,
                                              const int64_t* rows, const int64_t* cols, const double* scales,
                                              int32_t n_matrices, zero_muon_table** out) {
    using zero::fail;
    static const char* const who = "zero_muon_table_create";
    zero::clear_error();
    const std::string w(who);
    if (!out) return fail(ZERO_EINVAL, w + ": NULL out");
    *out = nullptr;
    if (n_matrices < 0) return fail(ZERO_EINVAL, w + ": n_matrices < 0");
    if (n_matrices > 0 && (!masters || !momenta || !grads || !params_out || !rows || !cols || !scales))
        return fail(ZERO_EINVAL, w + ": NULL array of pointers");
    zero_muon_table* tab = nullptr;
    try {
        std::vector<Desc> descs;
        std::vector<zero::Span> written, read;
        for (int32_t i = 0; i < n_matrices; ++i) {
            const std::string of = w + ": matrix " + std::to_string(i);
            if (rows[i] < 0 || cols[i] < 0) return fail(ZERO_EINVAL, of + " has a negative side");
            if (!std::isfinite(scales[i])) return fail(ZERO_EINVAL, of + " has a scale that is not finite");
            if (rows[i] == 0 || cols[i] == 0) continue;
            const zero_status st = check_sides(rows[i], cols[i], of);
            if (st != ZERO_OK) return st;
            Desc d{};
            d.src = grads[i];
            d.momentum = momenta[i];
            d.master = masters[i];
            d.out = params_out[i];
            d.scale = scales[i];
            if (!d.src || !d.momentum || !d.master || !d.out) return fail(ZERO_EINVAL, of + " has a NULL array");
            zero::muon::shape(&d, rows[i], cols[i], kTile);
            const size_t n = static_cast<size_t>(rows[i] * cols[i]);
            written.push_back({d.master, 4 * n, "master", i});
            written.push_back({d.momentum, 4 * n, "momentum", i});
            written.push_back({d.out, 2 * n, "param_out", i});
            read.push_back({d.src, 2 * n, "grad", i});
            descs.push_back(d);
        }
        const std::string clash = zero::copy::first_overlap_sorted(std::move(written), read);
        if (!clash.empty()) return fail(ZERO_EINVAL, w + ": " + clash);
        // The longest sums first: the tiles dispatched last are then the shortest.
        std::stable_sort(descs.begin(), descs.end(), [](const Desc& a, const Desc& b) {
            return int64_t(a.M) + a.N > int64_t(b.M) + b.N;
        });
        tab = new zero_muon_table;
        tab->descs = std::move(descs);
        const zero_status st = fill_table(tab, who);
        if (st != ZERO_OK) {
            zero_muon_table_free(tab);
            return st;
        }
    } catch (const std::bad_alloc&) {
        zero_muon_table_free(tab);
        return fail(ZERO_ENOMEM, w + ": host allocation failed");
    }
    *out = tab;
    return ZERO_OK;
}

extern "C" size_t zero_muon_table_workspace_bytes(const zero_muon_table* table) {
    return table ? static_cast<size_t>(table->bytes) : 0;
}

extern "C" int32_t zero_muon_table_matrices(const zero_muon_table* table) {
    return table ? static_cast<int32_t>(table->descs.size()) : -1;
}

extern "C" zero_status zero_muon_table_step(const zero_muon_table* table, double lr, double mu, int32_t nesterov,
                                            double weight_decay, const double* coefficients, int32_t n_steps,
                                            double eps, const float* clip_scale, void* workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
    using zero::fail;
    static const char* const who = "zero_muon_table_step";
    zero::clear_error();
    if (!table) return fail(ZERO_EINVAL, "zero_muon_table_step: NULL table");
    Call c{};
    zero_status st = muon_call(lr, mu, nesterov, weight_decay, coefficients, n_steps, eps, clip_scale, &c, who);
    if (st != ZERO_OK || table->descs.empty()) return st;
    int dev = -1;
    st = zero::check_hip(hipGetDevice(&dev), who);
    if (st != ZERO_OK) return st;
    if (dev != table->device)
        return fail(ZERO_EINVAL, std::string(who) + ": the table lives on device " + std::to_string(table->device) +
                                     ", the current device is " + std::to_string(dev));
    st = check_workspace(workspace, workspace_bytes, table->bytes, who);
    if (st != ZERO_OK) return st;
    const zero::Span ws{workspace, static_cast<size_t>(table->bytes), "workspace"};
    for (const Desc& d : table->descs) {
        const size_t n = static_cast<size_t>(d.rows) * static_cast<size_t>(d.cols);
        const zero::Span others[] = {
            {d.src, 2 * n, "grad"}, {d.momentum, 4 * n, "momentum"}, {d.master, 4 * n, "master"}, {d.out, 2 * n, "param_out"}};
        const std::string clash = zero::first_overlap(&ws, 1, others, 4);
        if (!clash.empty()) return fail(ZERO_EINVAL, std::string(who) + ": " + clash);
        add_cost(&c, d);
    }
    Matrices m = table->m;
    place(&m, workspace, table->partials);
    return launch(m, c, stream, who);
}
