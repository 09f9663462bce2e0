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
// orders of storage and padded with zeros, so that every product reads
// rows of contiguous K and needs no bounds checks), then the products, each one
// launch over the tiles of every matrix of the call; the last one's epilogue is
// the weight update.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "internal.hpp"
#include "muon_device.hpp"
#include "muon_short.hpp"
#include "pieces.hpp"

#pragma clang fp contract(off)

namespace {

using namespace zero::muon;
using namespace zero::muon::dev;

// Momentum and squared norm: each workgroup takes one chunk of one matrix. Bound by HBM: 10 bytes an element read and
// written at 5.3 TB/s (two 8192 x 8192: 254 us; a copy of 1 GB runs at 5.1).
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
    auto add = [&](int64_t i, int count) {
        float u[4];
        input4<kSource, true>(d, i, count, s, clip, u);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < count) sum += static_cast<double>(u[k]) * u[k];
    };
    int64_t i = lo + 4 * threadIdx.x;
#pragma unroll 2
    for (; i + 4 <= hi; i += 4 * kThreads) add(i, 4);
    if (i < hi) add(i, static_cast<int>(hi - i));
    sum = zero::dev::block_sum<kThreads>(sum, lds);
    if (threadIdx.x == 0) m.partials[d.first_partial + static_cast<int64_t>(c)] = sum;
}

__device__ __forceinline__ f16* buffer(const Matrices& m, const Desc& d, int32_t which) {
    const int64_t x = static_cast<int64_t>(d.M) * stride(d.N), xt = static_cast<int64_t>(d.N) * stride(d.M),
                  mm = static_cast<int64_t>(d.M) * stride(d.M);
    f16* const at = reinterpret_cast<f16*>(m.ws + d.ws);
    switch (which) {
        case zero::muon::kX: return at;
        case zero::muon::kT0: return at + x;
        case zero::muon::kT1: return at + x + xt;
        case zero::muon::kS0: return at + x + 2 * xt;
        case zero::muon::kS1: return at + x + 2 * xt + mm;
        case zero::muon::kS2: return at + x + 2 * xt + 2 * mm;
        default: return at + x + 2 * xt + 3 * mm;        // kLow
    }
}

// Packs a 64 x 64 tile of the padded matrix: u * 2^(13 - e), where |u| lies in [2^e, 2^(e + 1)), as fp16 in both
// orders, and with kLowPart what the rounding left. X is 2^-14 kappa times what is held. A thread holds 4 x 4 values;
// the other order goes through LDS, so that both are written in rows of 128 bytes. Bound by HBM: 12 bytes an element (u
// formed again from 6, three fp16 arrays written) at 4.9 TB/s (two 8192 x 8192: 324 us).
template <int kSource, bool kLowPart>
__global__ __launch_bounds__(kThreads) void pack_kernel(Matrices m, MomentumScalars s, double eps) {
    __shared__ f16x4 turned[kLowPart ? 2 : 1][kPack * kPack / 4];
    __shared__ double lds[kThreads / zero::dev::kWave];
    __shared__ double total;
    if (skipped(s.clip)) return;
    const float clip = s.clip != nullptr ? *s.clip : 1.0f;
    uint32_t t;
    const Desc d = find(m, zero::muon::kByPack, blockIdx.x, &t);
    // The source's rows run along `tall ? N : M`.
    const bool tall = d.rows > d.cols;
    const int32_t padded_rows = tall ? d.N : d.M, padded_cols = tall ? d.M : d.N;
    const uint32_t tiles = padded_cols / kPack;
    const int32_t r0 = static_cast<int32_t>(t / tiles) * kPack, c0 = static_cast<int32_t>(t % tiles) * kPack;
    const int down = threadIdx.x / 16, right = threadIdx.x % 16;       // the thread's 4 x 4 values
    float x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int32_t r = r0 + down * 4 + k, c = c0 + right * 4;
        int n = r < d.rows ? d.cols - c : 0;
        n = n < 0 ? 0 : n > 4 ? 4 : n;
        input4<kSource, false>(d, static_cast<int64_t>(r) * d.cols + c, n, s, clip, x[k]);
    }
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

    f16x4 high[4], low[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = ldexpf(x[k][j], 13 - e);
        split4(x[k][0], x[k][1], x[k][2], x[k][3], &high[k], &low[k]);
    }
    f16* const along = buffer(m, d, tall ? zero::muon::kT0 : zero::muon::kX);
    f16* const across = buffer(m, d, tall ? zero::muon::kX : zero::muon::kT0);
    f16* const rest = buffer(m, d, zero::muon::kLow);                  // as `across`
    // Column 4 right + j of the tile, its piece `down` of four rows, at place down ^ right.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        turned[0][(right * 4 + j) * 16 + (down ^ right)] = f16x4{high[0][j], high[1][j], high[2][j], high[3][j]};
        if constexpr (kLowPart)
            turned[1][(right * 4 + j) * 16 + (down ^ right)] = f16x4{low[0][j], low[1][j], low[2][j], low[3][j]};
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t at = static_cast<int64_t>(r0 + down * 4 + k) * stride(padded_cols) + c0 + right * 4;
        *reinterpret_cast<f16x4*>(along + at) = high[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = down + k * 16;
        const int64_t at = static_cast<int64_t>(c0 + c) * stride(padded_rows) + r0 + right * 4;
        *reinterpret_cast<f16x4*>(across + at) = turned[0][c * 16 + (right ^ (c / 4))];
        if constexpr (kLowPart)
            *reinterpret_cast<f16x4*>(rest + at) = turned[1][c * 16 + (right ^ (c / 4))];
    }
}

// A product's tile: kRows x kCols waves, each of MI x NI MFMA tiles of kSide x kSide, kInner deep. (A chip full of MFMAs is
// limited by its power: from registers alone 16 x 16 x 32 sustains 1905 TFLOP/s and 32 x 32 x 16, which reads its
// accumulators twice as often, 1640.)
constexpr int kRows = 2, kCols = 2, kWaves = kRows * kCols;
constexpr int kSide = 16, kInner = 32;

// K elements of one LDS stage: a row's 128 bytes are one cache line. One stage is multiplied, the others are on their
// way.
constexpr int kDepth = 64;

// A stage's rows hold eight 16-byte pieces, piece p of row r at place p ^ (r / 2 % 8): 16 rows' pieces of one column
// then lie in all banks.
__device__ __forceinline__ int swizzle(int r, int p) { return p ^ ((r >> 1) & 7); }

typedef __attribute__((address_space(3))) void lds_void;

// Waits for the wave's LDS reads and until at most n of its loads are on their way, then for the workgroup.
template <int n>
__device__ __forceinline__ void landed_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(n) : "memory");
}

// Tile t of a matrix of `rows` x `cols` tiles, in strips of kStrip rows, column by column within a strip: 32 tiles
// in order share 4 rows' and 8 columns' panels.
constexpr int32_t kStrip = 4;

__device__ __forceinline__ void rect_tile(uint32_t t, int32_t rows, int32_t cols, int32_t* bi, int32_t* bj) {
    const uint32_t strip = t / (kStrip * cols), first = strip * kStrip;
    const uint32_t in = t - strip * (kStrip * cols);
    const uint32_t h = rows - first < kStrip ? rows - first : kStrip;
    *bj = static_cast<int32_t>(in / h);
    *bi = static_cast<int32_t>(first + (in - *bj * h));
}

// The same of the lower triangle of `rows` x `rows` tiles.
__device__ __forceinline__ void triangle_tile(uint32_t t, int32_t rows, int32_t* bi, int32_t* bj) {
    int32_t i = static_cast<int32_t>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (static_cast<uint32_t>(i) * (i + 1) / 2 > t) --i;
    while (static_cast<uint32_t>(i + 1) * (i + 2) / 2 <= t) ++i;
    const int32_t first = i / kStrip * kStrip, h = rows - first < kStrip ? rows - first : kStrip;
    int32_t in = static_cast<int32_t>(t - static_cast<uint32_t>(first) * (first + 1) / 2);
    const int32_t whole = h * (first + 1);               // columns up to the diagonal's first
    if (in < whole) {
        *bj = in / h;
        *bi = first + (in - *bj * h);
        return;
    }
    in -= whole;
    int32_t left = h - 1, c = first + 1;
    while (in >= left) {
        in -= left;
        --left;
        ++c;
    }
    *bj = c;
    *bi = c + in;
}

// The tile of a workgroup: the dispatcher deals workgroups round-robin to the 8 XCDs, each with an L2 of its own, so
// runs of `run` tiles go to one XCD. (The grid is rounded up to whole runs on every XCD.)
__device__ __forceinline__ uint32_t xcd_tile(uint32_t run) {
    const uint32_t x = blockIdx.x % 8, s = blockIdx.x / 8;
    return (s / run * 8 + x) * run + s % run;
}

// Where a tile lies: its first row and column, how many of them another tile writes, and whether it is also written
// mirrored.
struct Place {
    int32_t r0, c0, skip_rows, skip_cols;
    bool mirror;
};

// Whether a product's last tiles can be cut into quarters.
template <int T, bool kSquareOut>
constexpr bool has_quarters = T == 256 && kSquareOut;

// One T x T tile of a product, both operands rows of contiguous K.
//
// With 256 the MFMAs bound it and the chip's power their clock: without what carrying the roundings adds to the epilogue two
// applies of 8192 x 8192 x 8192 take 1.60 ms, 1375 TFLOP/s (the library's product of that size 1395), the MFMAs busy 71 % of the
// time at 1.84 GHz (2048 of a stage's 2,800 cycles; its loads, 64 KB into one compute unit's LDS, need 1024), with it
// 1.79 to 1.86 ms. Symmetric products run at 1.2 PFLOP/s, half of each computed. Where the tiles are few (487 x 1000: 36 of 64 x 64, 7.2 us a product) it is latency: 1.4 us of launch,
// 1 to the first load, 2.4 for eight stages, 1.8 for the way out through LDS. Rows of K come straight from memory to
// LDS (16 bytes a lane), so that no register holds what is on its way.
template <int T, int kStages, bool kSquareOut, int kEnd>     // kEnd: 0 workspace, 1 orthogonalised matrix, 2 weight update
__device__ __forceinline__ void tile(const Matrices& m, const Product& p, const Update& u, const Desc& d, const Place& at_place,
                                     f16* lds) {
    constexpr int MI = T / kSide / kRows, NI = T / kSide / kCols;
    constexpr int kOperand = T * kDepth;                 // values of one operand's stage
    constexpr int kLoads = T / 8 / kWaves;               // of 8 rows each, a wave and operand
    const int32_t r0 = at_place.r0, c0 = at_place.c0, skip_rows = at_place.skip_rows, skip_cols = at_place.skip_cols;
    const bool tall = d.rows > d.cols;
    const int32_t height = tall ? d.N : d.M;             // of an apply's output
    const int32_t K = p.kind == Kind::kGram ? d.N : d.M, ld = stride(K);
    const f16* left = buffer(m, d, p.lhs);
    const f16* right = buffer(m, d, p.rhs);
    if (!kSquareOut && tall) {            // rows of the output are the source's: X^T on the left
        const f16* const x = left;
        left = right;
        right = x;
    }
    left += static_cast<int64_t>(r0) * ld;
    right += static_cast<int64_t>(c0) * ld;

    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wr = wave / kCols * (MI * kSide), wc = wave % kCols * (NI * kSide);

    // Global to LDS: lane l of a load brings the piece that belongs at place l % 8 of row l / 8.
    const int32_t all = K / kDepth;
    __amdgpu_buffer_rsrc_t from[2] = {zero::dev::through_rsrc(left), zero::dev::through_rsrc(right)};
    uint32_t at[kLoads];
    const int row = lane / 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (wave * kLoads + i) * 8 + row;
        at[i] = static_cast<uint32_t>(r) * ld * 2 + swizzle(r, lane % 8) * 16;
    }
    // Load q of stage s: the left operand's kLoads, then the right's.
    auto load = [&](int32_t s, int q) {
        f16* const to = lds + (s % kStages) * 2 * kOperand;
        const uint32_t k = static_cast<uint32_t>(s) * (kDepth * 2);
        const int o = q / kLoads, i = q % kLoads;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            from[o], (lds_void*)(to + o * kOperand + (wave * kLoads + i) * 8 * kDepth), 16, at[i], k, 0, 0);
    };
    auto load_all = [&](int32_t s) {
#pragma unroll
        for (int q = 0; q < 2 * kLoads; ++q) load(s, q);
    };
    const int turn = (lane % kSide) >> 1;                // of the lane's rows in a fragment
    const int a_row = (wr + lane % kSide) * kDepth, b_row = kOperand + (wc + lane % kSide) * kDepth;
    f32x4 acc[MI][NI] = {};
    auto keep_sums = [&] {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    struct Fragments {
        f16x8 a[MI], b[NI];
    };
    // Read r of the fragments of K elements 32 kk to 32 kk + 31 of stage s.
    auto read = [&](int32_t s, int kk, int r, Fragments& f) {
        const f16* const st = lds + (s % kStages) * 2 * kOperand + ((4 * kk + lane / kSide) ^ turn) * 8;
        if (r < MI)
            f.a[r] = *reinterpret_cast<const f16x8*>(st + a_row + r * kSide * kDepth);
        else
            f.b[r - MI] = *reinterpret_cast<const f16x8*>(st + b_row + (r - MI) * kSide * kDepth);
    };
    constexpr int kReads = MI + NI, kProducts = MI * NI;
    // In assembly, so that the sum stays where it is: the compiler may give the result of this shape other registers, and
    // with 256 of them moves them all in every stage. (A product that adds to the one before needs no wait. The wait between the
    // last product and the first read of a sum, which the compiler puts after its own instruction, stands behind the loop.)
    auto multiply = [&](const Fragments& f, int q) {
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc[q / NI][q % NI]) : "v"(f.a[q / NI]), "v"(f.b[q % NI]));
    };
    keep_sums();                                         // set to 0, and two cycles before the first product
    asm volatile("s_nop 3" ::: "memory");
    if constexpr (kStages == 2) {
        // A stage is two phases of MI * NI products, and between these are issued, in this order, the reads of the next
        // phase's fragments and the loads of stage s + 2: in a row they would hold the products up. At the barrier all
        // waves have read stage s, whose place stage s + 2 takes, and stage s + 1 has landed for every wave; its loads had
        // the other quarter of a stage to. (8192 x 8192, 128 stages: the loads spread over half a stage 1 % slower, over
        // a quarter 7 %; four stages of half the depth, with twice the barriers, 6 %.)
        Fragments f0, f1;
        static_assert(kDepth == 2 * kInner, "two phases");
        constexpr int kFree = kProducts * 3 / 4, kSpread = 2 * kProducts - kFree;
        auto stage = [&](int32_t s, auto load_next) {
            constexpr int kCount = load_next ? 2 * kLoads : 0;
            int loads = 0;
            auto phase = [&](const Fragments& now, Fragments& next, int32_t from_stage, int kk, int first) {
                int reads = 0;
#pragma unroll
                for (int q = 0; q < kProducts; ++q) {
                    const int at = first + q - kFree;    // products since the barrier
                    if (at == 0) landed_and_barrier<0>();
                    multiply(now, q);
#pragma unroll
                    for (; reads * kProducts < (q + 1) * kReads * 2 && reads < kReads; ++reads) read(from_stage, kk, reads, next);
#pragma unroll
                    for (; loads * kSpread < (at + 1) * kCount; ++loads) load(s + 2, loads);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            phase(f0, f1, s, 1, 0);
            phase(f1, f0, s + 1, 0, kProducts);          // (what it reads after the last stage is not used)
        };
        load_all(0);
        if (1 < all) load_all(1);
        if (1 < all)
            landed_and_barrier<2 * kLoads>();
        else
            landed_and_barrier<0>();
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(0, 0, r, f0);
        int32_t s = 0;
        for (; s + 2 < all; ++s) stage(s, std::true_type{});
        for (; s < all; ++s) stage(s, std::false_type{});
    } else {
        // With few products between two reads their latency would show at each phase: all fragments of stage s + 1 are read
        // while stage s multiplies. At a stage's barrier stage s + 1 has landed for every wave, and every wave has
        // read all of stage s, whose place stage s + kStages takes.
        constexpr std::integral_constant<int, (kStages - 2) * 2 * kLoads> kFlying{};
        constexpr int kPhases = kDepth / kInner;
        Fragments f0[kPhases], f1[kPhases];
        auto stage = [&](int32_t s, const Fragments* now, Fragments* next) {
            if (s + kStages <= all)
                landed_and_barrier<kFlying>();           // stages s + 2 to s + kStages - 1 may fly
            else
                landed_and_barrier<0>();
            if (s + kStages < all) load_all(s + kStages);
            int reads = 0;
#pragma unroll
            for (int at = 0; at < kPhases * kProducts; ++at) {
                multiply(now[at / kProducts], at % kProducts);
#pragma unroll
                for (; reads * kProducts < (at + 1) * kReads * 2 && reads < kPhases * kReads; ++reads)
                    read(s + 1, reads / kReads, reads % kReads, next[reads / kReads]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            if (s < all) load_all(s);
        if (all >= kStages)
            landed_and_barrier<(kStages - 1) * 2 * kLoads>();
        else
            landed_and_barrier<0>();
#pragma unroll
        for (int kk = 0; kk < kPhases; ++kk)
#pragma unroll
            for (int r = 0; r < kReads; ++r) read(0, kk, r, f0[kk]);
        int32_t s = 0;
        for (; s + 1 < all; s += 2) {
            stage(s, f0, f1);
            stage(s + 1, f1, f0);
        }
        if (s < all) stage(s, f0, f1);                   // (what the last one reads is not used)
    }

    // A sum may be read eight wait states after its last product (the compiler's own distance); these are 32.
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    keep_sums();

    // A lane holds one column of each MFMA tile, four consecutive rows at a time; LDS turns them into whole rows, in
    // either order of storage, so that memory is read and written 16 bytes a lane and 2 T bytes a row.
    float alpha = p.alpha;
    if (p.kappa_power > 0) {
        const float kappa = m.kappa[d.id];
        alpha = p.kappa_power == 2 ? alpha * (kappa * kappa) : alpha * kappa;
    }
    const int down = wr + lane / kSide * 4, over = wc + lane % kSide;  // the lane's first row, and its column
    const int quad = lane % 4;
    // Where eight bytes lie: four values of row r from column 4 g. Rows that are close lie in other banks.
    auto place = [&](int r, int g) {
        const int turned = T % 128 == 0 || T == 64 ? (2 * r) & (T / 8 - 1) : (r >> 1) & 7;
        return r * T + (((g >> 1) ^ turned) << 3) + (g & 1) * 4;
    };
    // A thread's 16-byte pieces: kGroup threads, a power of two, hold pieces next to each other of one row.
    constexpr int kPerRow = T / 8, kGroup = kPerRow & -kPerRow, kAcross = kPerRow / kGroup;
    constexpr int kRowStep = 64 * kWaves / kGroup, kOwn = T / kRowStep * kAcross;
    auto row_of = [&](int k) { return static_cast<int>(threadIdx.x) / kGroup + k / kAcross * kRowStep; };
    auto piece_of = [&](int k) { return static_cast<int>(threadIdx.x) % kGroup + k % kAcross * kGroup; };
    // The tile in LDS to rows of `ld` values at `to`, but for what another tile writes.
    auto write_rows = [&](f16* to, int64_t ld, int32_t first_row, int32_t first_col) {
        constexpr int kAtOnce = kOwn < 8 ? kOwn : kOwn % 8 == 0 ? 8 : 6;
        static_assert(kOwn % kAtOnce == 0, "whole groups");
#pragma unroll 1
        for (int k0 = 0; k0 < kOwn; k0 += kAtOnce) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int r = row_of(k0 + k), piece = piece_of(k0 + k);
                if (r >= first_row && piece * 8 >= first_col)
                    *reinterpret_cast<f16x8*>(to + r * ld + piece * 8) =
                        *reinterpret_cast<const f16x8*>(lds + place(r, piece * 2));
            }
        }
    };
    // And `from` there, each piece as change(piece, row, number) makes it.
    auto read_rows = [&](const f16* from, int64_t ld, auto change) {
        constexpr int kAtOnce = kOwn < 8 ? kOwn : kOwn % 8 == 0 ? 8 : 6;
#pragma unroll 1
        for (int k0 = 0; k0 < kOwn; k0 += kAtOnce) {
            f16x8 x[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                x[k] = *reinterpret_cast<const f16x8*>(from + row_of(k0 + k) * ld + piece_of(k0 + k) * 8);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                *reinterpret_cast<f16x8*>(lds + place(row_of(k0 + k), piece_of(k0 + k) * 2)) =
                    change(x[k], row_of(k0 + k), piece_of(k0 + k));
        }
    };
    // Calls f(i, j) for the lane's groups of four rows.
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) f(i, j);
    };
    f16x4 values[MI][NI];
    // Q's diagonal times what rounding X left, both as fp16 times a power of two: their product needs no more bits. (In rows
    // and columns that a tile shares with the one before, that one may have written its own by now: what this one makes of
    // them is not stored.)
    f16* const q = lds + kStages * 2 * kOperand;         // 2^-14 of it
    if constexpr (!kSquareOut)
        if (p.low_in) {
            const int64_t step = stride(d.M) + 1;
            const f16* const diagonal = buffer(m, d, p.lhs) + (tall ? c0 : r0) * step;
            for (int k = threadIdx.x; k < T; k += 64 * kWaves) q[k] = diagonal[k * step] * static_cast<f16>(0x1p-14f);
        }
    __syncthreads();
    if constexpr (!kSquareOut)
        if (p.low_in) {
            const int64_t low_ld = stride(height);
            read_rows(buffer(m, d, zero::muon::kLow) + c0 * low_ld + r0, low_ld, [&](f16x8 x, int r, int piece) {
                if (!tall) return x * *reinterpret_cast<const f16x8*>(q + piece * 8);
                return x * q[r];
            });
            __syncthreads();
            each([&](int i, int j) {
                const f16x4 x = *reinterpret_cast<const f16x4*>(lds + place(over + j * kSide, (down + i * kSide) / 4));
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][j][k] += 0x1p14f * static_cast<float>(x[k]);
            });
            __syncthreads();
        }
    if constexpr (kSquareOut) {
        f16* const out = buffer(m, d, p.out);
        const int64_t ldm = stride(d.M);
        const int64_t direct = r0 * ldm + c0, mirrored = c0 * ldm + r0;
        if (p.add != zero::muon::kNone) {                // symmetric: its mirrored tile's rows are this one's columns
            read_rows(buffer(m, d, p.add) + mirrored, ldm, [](f16x8 x, int, int) { return x; });
            __syncthreads();
        }
        const int diagonal = c0 - r0 + over - down;               // row minus `down` of the lane's first column
        each([&](int i, int j) {
            f16x4 old = {};
            if (p.add != zero::muon::kNone)
                old = *reinterpret_cast<const f16x4*>(lds + place(over + j * kSide, (down + i * kSide) / 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x = alpha * acc[i][j][k] + p.beta * static_cast<float>(old[k]);
                if (i * kSide + k == diagonal + j * kSide) x += p.diag;
                values[i][j][k] = static_cast<f16>(x);
            }
        });
        if (p.add != zero::muon::kNone) __syncthreads();
        if (at_place.mirror) {
            each([&](int i, int j) {
                *reinterpret_cast<f16x4*>(lds + place(over + j * kSide, (down + i * kSide) / 4)) = values[i][j];
            });
            __syncthreads();
            write_rows(out + mirrored, ldm, skip_cols, skip_rows);
            __syncthreads();
        }
        each([&](int i, int j) {
            *reinterpret_cast<f16x4*>(lds + place(down + i * kSide + quad, (over + j * kSide) / 4)) =
                quad_transpose(values[i][j]);
        });
        __syncthreads();
        write_rows(out + direct, ldm, skip_rows, skip_cols);
    } else if constexpr (kEnd == 0) {
        const int64_t down_ld = stride(tall ? d.N : d.M), along_ld = stride(tall ? d.M : d.N);
        f16* const along = buffer(m, d, tall ? p.out_t : p.out);
        f16* const across = buffer(m, d, tall ? p.out : p.out_t);
        // What rounding leaves first, then the rounded values, formed again: both do not fit the registers.
        if (p.low_out) {
            each([&](int i, int j) {
                f16x4 x, rest;
                split4(alpha * acc[i][j][0], alpha * acc[i][j][1], alpha * acc[i][j][2], alpha * acc[i][j][3], &x, &rest);
                *reinterpret_cast<f16x4*>(lds + place(over + j * kSide, (down + i * kSide) / 4)) = rest;
            });
            __syncthreads();
            write_rows(buffer(m, d, zero::muon::kLow) + c0 * down_ld + r0, down_ld, skip_cols, skip_rows);
            __syncthreads();
        }
        each([&](int i, int j) {
            f16x4 rest;
            split4(alpha * acc[i][j][0], alpha * acc[i][j][1], alpha * acc[i][j][2], alpha * acc[i][j][3], &values[i][j], &rest);
            *reinterpret_cast<f16x4*>(lds + place(over + j * kSide, (down + i * kSide) / 4)) = values[i][j];
        });
        __syncthreads();
        write_rows(across + c0 * down_ld + r0, down_ld, skip_cols, skip_rows);
        __syncthreads();
        each([&](int i, int j) {
            *reinterpret_cast<f16x4*>(lds + place(down + i * kSide + quad, (over + j * kSide) / 4)) =
                quad_transpose(values[i][j]);
        });
        __syncthreads();
        write_rows(along + r0 * along_ld + c0, along_ld, skip_rows, skip_cols);
    } else {
        // The orthogonalised matrix in bf16, as bits.
        each([&](int i, int j) {
            typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
            const u32x2_t bits = {zero::dev::pack_bf16(alpha * acc[i][j][0], alpha * acc[i][j][1]),
                                  zero::dev::pack_bf16(alpha * acc[i][j][2], alpha * acc[i][j][3])};
            *reinterpret_cast<f16x4*>(lds + place(down + i * kSide + quad, (over + j * kSide) / 4)) =
                quad_transpose(__builtin_bit_cast(f16x4, bits));
        });
        __syncthreads();
        const float rate = static_cast<float>(u.lr * d.scale);
        // Four pieces' loads before the first is used; only the last tiles of a matrix need the guards.
        constexpr int kAtOnce = kOwn < 4 ? kOwn : kOwn % 4 == 0 ? 4 : 3;
        static_assert(kOwn % kAtOnce == 0, "whole groups");
#pragma unroll 1
        for (int k0 = 0; k0 < kOwn; k0 += kAtOnce) {
            float w[kAtOnce][8];
            int64_t first[kAtOnce];
            int here[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int r = row_of(k0 + k), piece = piece_of(k0 + k);
                const int32_t c = c0 + piece * 8;
                first[k] = static_cast<int64_t>(r0 + r) * d.cols + c;
                const bool own = r >= skip_rows && piece * 8 >= skip_cols && r0 + r < d.rows && c < d.cols;
                here[k] = !own ? 0 : d.cols - c < 8 ? d.cols - c : 8;
                if constexpr (kEnd == 2) {
                    read4(d.master, first[k], here[k] < 4 ? here[k] : 4, w[k]);
                    read4(d.master, first[k] + 4, here[k] < 4 ? 0 : here[k] - 4, w[k] + 4);
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const f16x8 o = *reinterpret_cast<const f16x8*>(lds + place(row_of(k0 + k), piece_of(k0 + k) * 2));
                uint16_t bits[8];
                __builtin_memcpy(bits, &o, sizeof(bits));
                finish8<kEnd>(d, u, rate, first[k], here[k], bits, w[k]);
            }
        }
    }
}

// The tile of a workgroup. Tiles from `whole` on, the few that a last round of 256 x 256 would be for, are cut into
// quarters, each a workgroup's (a side of 8192 has 528 tiles, of which 512 fill two rounds: 570 to 510 us at K 8192).
template <int T, int kStages, bool kSquareOut, int kEnd>
__device__ __forceinline__ void product(const Matrices& m, const Product& p, const Update& u, uint32_t run, uint32_t whole) {
    constexpr int kValues = kStages * 2 * T * kDepth;    // values of all stages
    // (With an apply's diagonal of Q behind them: an array of its own makes the compiler wait for all loads on their way to
    // LDS before it reads the fragments, 2.9 ms more for two applies of 8192 x 8192 x 8192.)
    __shared__ __align__(16) f16 lds[kValues + (kSquareOut ? 0 : T)];
    static_assert(kValues >= T * T, "the tile fits where the stages were");
    if (kEnd == 2 && skipped(u.clip)) return;
    uint32_t t = xcd_tile(run), quarter = 0;
    const bool full = kSquareOut && p.full;              // two workgroups for a tile and the one mirrored to it
    const bool above = full && t % 2 != 0;
    if (full) t /= 2;
    const bool cut = has_quarters<T, kSquareOut> && !full && t >= whole;
    if (cut) {
        quarter = (t - whole) % 4;
        t = whole + (t - whole) / 4;
    }
    constexpr int kGrid = kSquareOut ? zero::muon::kByPair : zero::muon::kByTile;
    if (t >= m.total[kGrid]) return;
    const Desc d = find(m, kGrid, t, &t);
    const bool tall = d.rows > d.cols;
    const int32_t height = !kSquareOut && tall ? d.N : d.M, width = kSquareOut || tall ? d.M : d.N;
    int32_t bi, bj;
    if constexpr (kSquareOut)
        triangle_tile(t, (height + T - 1) / T, &bi, &bj);
    else
        rect_tile(t, (height + T - 1) / T, (width + T - 1) / T, &bi, &bj);
    if (above) {
        if (bi == bj) return;
        const int32_t swapped = bi;
        bi = bj;
        bj = swapped;
    }
    // The last tiles end with the matrix; the rows and columns that they share with the tiles before are those tiles'.
    Place at;
    at.r0 = min(bi * T, height - T);
    at.c0 = min(bj * T, width - T);
    at.skip_rows = bi * T - at.r0;
    at.skip_cols = bj * T - at.c0;
    at.mirror = !full && bi != bj;
    if constexpr (has_quarters<T, kSquareOut>) {
        if (cut) {
            constexpr int kHalf = T / 2;
            const int32_t down = quarter / 2 * kHalf, right = quarter % 2 * kHalf;
            if (bi == bj && down < right) return;        // the one below the diagonal is mirrored there
            if (at.skip_rows >= down + kHalf || at.skip_cols >= right + kHalf) return;
            at.r0 += down;
            at.c0 += right;
            at.skip_rows = max(at.skip_rows - down, 0);
            at.skip_cols = max(at.skip_cols - right, 0);
            at.mirror = at.mirror || down != right;
            return tile<kHalf, kStages, kSquareOut, kEnd>(m, p, u, d, at, lds);
        }
    }
    tile<T, kStages, kSquareOut, kEnd>(m, p, u, d, at, lds);
}

template <int T, int kStages, bool kSquareOut, int kEnd>
__global__ __launch_bounds__(64 * kWaves) void product_kernel(Matrices m, Product p, Update u, uint32_t run, uint32_t whole) {
#ifdef __HIP_DEVICE_COMPILE__                            // the host has no such instructions
    product<T, kStages, kSquareOut, kEnd>(m, p, u, run, whole);
#endif
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
    zero::muon::Times times;
};

template <int T, int kStages, bool kSquareOut, int kEnd>
void launch_product(const Matrices& m, const Product& p, const Update& u, hipStream_t stream) {
    // Whole runs on every XCD; no run longer than an eighth of the tiles, so that a short grid reaches every XCD.
    const uint32_t tiles = m.total[kSquareOut ? zero::muon::kByPair : zero::muon::kByTile];
    const bool full = kSquareOut && p.full;
    const uint32_t whole = has_quarters<T, kSquareOut> && !full ? zero::muon::whole_tiles(tiles) : tiles;
    const uint32_t total = full ? 2 * tiles : whole + 4 * (tiles - whole);
    const uint32_t run = std::min(32u, (total + 7) / 8);
    const uint32_t blocks = (total + 8 * run - 1) / (8 * run) * (8 * run);
    hipLaunchKernelGGL((product_kernel<T, kStages, kSquareOut, kEnd>), dim3(blocks),
                       dim3(64 * kWaves), 0, stream, m, p, u, run, whole);
}

template <bool kSquareOut, int kEnd>
void launch_product(const Matrices& m, const Product& p, const Update& u, hipStream_t stream) {
    const int64_t tile = kSquareOut ? m.square_tile : m.rect_tile;
    if (tile == 64) {
        // More stages on their way where they cost no third workgroup on a compute unit. (Kernel times of five steps:
        // 487 x 1000 takes 143 us with four stages and 152 with three, six matrices of a 124 M GPT 447 and 414.)
        const uint32_t total = m.total[kSquareOut ? zero::muon::kByPair : zero::muon::kByTile];
        if (total <= 2 * zero::muon::kUnits) return launch_product<64, 4, kSquareOut, kEnd>(m, p, u, stream);
        return launch_product<64, 3, kSquareOut, kEnd>(m, p, u, stream);
    }
    if (tile == 128) return launch_product<128, 2, kSquareOut, kEnd>(m, p, u, stream);
    if constexpr (kSquareOut)
        if (tile == 192) return launch_product<192, 2, kSquareOut, kEnd>(m, p, u, stream);
    launch_product<256, 2, kSquareOut, kEnd>(m, p, u, stream);
}

template <int kSource, int kEnd>
zero_status launch_all(const Matrices& m, const Call& c, const std::vector<Product>& program, hipStream_t stream,
                       const char* who) {
    hipLaunchKernelGGL(momentum_kernel<kSource>, dim3(m.total[zero::muon::kByChunk]), dim3(kThreads), 0, stream, m,
                       c.momentum);
    zero_status st = zero::check_hip(hipGetLastError(), who);
    if (st != ZERO_OK) return st;
    hipLaunchKernelGGL((pack_kernel<kSource, kSource != 0>), dim3(m.total[zero::muon::kByPack]), dim3(kThreads), 0,
                       stream, m, c.momentum, c.eps);
    st = zero::check_hip(hipGetLastError(), who);
    for (const Product& p : program) {
        if (st != ZERO_OK) return st;
        if (p.kind == Kind::kGram || p.kind == Kind::kSquare)
            launch_product<true, 0>(m, p, c.update, stream);
        else if (p.kind == Kind::kApply)
            launch_product<false, 0>(m, p, c.update, stream);
        else
            launch_product<false, kEnd>(m, p, c.update, stream);
        st = zero::check_hip(hipGetLastError(), who);
    }
    return st;
}

zero_status launch(const Matrices& m, const Call& c, hipStream_t stream, const char* who) {
    ShortProgram steps;
    if (m.side != 0 && make_short_program(c.coefficients, c.n_steps, &steps))
        return launch_short(c.source, m, c.momentum, c.update, steps, c.eps, stream, who);
    std::vector<Product> program;
    // Pairs where they save a fiftieth of the time or more (six GPT-2 small matrices: 404 us against 429; 487 x 1000: 130
    // against 127): at equal time the single steps, whose A comes from X itself, are more exact (up to 4.7e-3 of the result's
    // norm on hard singular values against 6.1e-3).
    const bool pairs = zero::muon::program_time(c.times, c.n_steps, true) <
                       0.98 * zero::muon::program_time(c.times, c.n_steps, false);
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

constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / 512 - 256;         // fewer than 2^32 work-items a launch of twice as many

// A stack's sizes: its first matrix's descriptor (sides, chunks), the workgroups, the products' times and the workspace.
// ZERO_ERANGE where one launch does not hold it.
zero_status measure_stack(int64_t count, int64_t rows, int64_t cols, Matrices* m, zero::muon::Times* times, int64_t* bytes,
                          const char* who) {
    zero_status st = check_sides(rows, cols, who);
    if (st != ZERO_OK) return st;
    zero::muon::TileChoice choice;
    choice.add(count, rows, cols);
    choice.best(&m->square_tile, &m->rect_tile, times);
    zero::muon::shape(&m->base, rows, cols, std::max(m->square_tile, m->rect_tile));
    m->side = short_side(std::min(rows, cols));
    m->base.parts = m->side != 0 ? short_parts(m->side, std::max(rows, cols), count) : 1;
    m->numel = rows * cols;
    m->area = zero::muon::area_bytes(m->base);
    for (int g = 0; g < kGrids; ++g) {
        const int64_t per = zero::muon::grid_count(m->base, g, m->square_tile, m->rect_tile);
        if (count > kMaxBlocks / per)
            return zero::fail(ZERO_ERANGE, std::string(who) + ": more workgroups than one launch holds");
        m->per[g] = static_cast<uint32_t>(per);
        m->total[g] = static_cast<uint32_t>(per * count);
    }
    m->matrices = static_cast<uint32_t>(count);
    const int64_t head = zero::muon::head_bytes(count * m->base.chunks, count);
    if (count > (INT64_MAX - head) / m->area) return zero::fail(ZERO_ERANGE, std::string(who) + ": workspace overflows");
    *bytes = head + count * m->area;
    m->base.ws = head;
    if (m->side != 0) {
        m->base.short_ws = short_head_bytes(m->total[kByPart], count);
        m->short_area = short_area_bytes(m->side, m->base.parts);
        *bytes = std::max(*bytes, m->base.short_ws + count * m->short_area);
    }
    return ZERO_OK;
}

void place(Matrices* m, void* workspace, int64_t partials) {
    m->ws = static_cast<char*>(workspace);
    m->part_exponent = static_cast<int32_t*>(workspace);
    m->short_scale = reinterpret_cast<ShortScale*>(m->ws + short_scales_at(m->total[kByPart]));
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

}  // namespace

extern "C" size_t zero_muon_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
    Matrices m{};
    int64_t bytes = 0;
    bool empty = false;
    zero::muon::Times times;
    if (check_counts(count, rows, cols, &empty, "zero_muon_workspace_bytes") != ZERO_OK || empty) return 0;
    if (measure_stack(count, rows, cols, &m, &times, &bytes, "zero_muon_workspace_bytes") != ZERO_OK) return 0;
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
    Call c{};
    int64_t need = 0;
    st = measure_stack(count, rows, cols, &m, &c.times, &need, who);
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
    c.coefficients = coefficients;
    c.n_steps = n_steps;
    c.eps = eps;
    c.source = x_type == ZERO_MATRIX_F32 ? 1 : 0;
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
    st = measure_stack(count, rows, cols, &m, &c.times, &need, who);
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
    return launch(m, c, stream, who);
}

// ------------------------------------------------------------ a list of matrices

struct zero_muon_table {
    void* mem = nullptr;              // descriptors, then the grids' indexes
    int device = -1;
    std::vector<Desc> descs;
    Matrices m{};
    int64_t partials = 0;
    int64_t bytes = 0;                // of the workspace
    zero::muon::Times times{};
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
    zero::muon::TileChoice choice;
    for (const Desc& d : tab->descs) choice.add(1, d.rows, d.cols);
    choice.best(&tab->m.square_tile, &tab->m.rect_tile, &tab->times);
    int64_t most = 0;
    for (const Desc& d : tab->descs) most = std::max<int64_t>(most, std::min(d.rows, d.cols));
    tab->m.side = short_side(most);
    tab->m.matrices = static_cast<uint32_t>(tab->descs.size());
    for (Desc& d : tab->descs) {
        zero::muon::shape(&d, d.rows, d.cols, std::max(tab->m.square_tile, tab->m.rect_tile));
        d.parts = tab->m.side != 0 ? short_parts(tab->m.side, std::max(d.rows, d.cols), tab->m.matrices) : 1;
    }
    std::vector<uint32_t> index;
    size_t starts[kGrids] = {};
    for (int g = 0; g < kGrids; ++g) {
        starts[g] = index.size();
        int64_t total = 0;
        for (size_t i = 0; i < tab->descs.size(); ++i) {
            Desc& d = tab->descs[i];
            const int64_t n = zero::muon::grid_count(d, g, tab->m.square_tile, tab->m.rect_tile);
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
    if (tab->m.side != 0) {
        int64_t bytes = short_head_bytes(tab->m.total[kByPart], tab->m.matrices);
        for (Desc& d : tab->descs) {
            d.short_ws = bytes;
            bytes += short_area_bytes(tab->m.side, d.parts);
        }
        tab->bytes = std::max(tab->bytes, bytes);
    }
    zero_status st = zero::check_hip(hipGetDevice(&tab->device), "zero_muon_table_create: hipGetDevice");
    if (st != ZERO_OK) return st;
    const size_t table_bytes = tab->descs.size() * sizeof(Desc), index_bytes = index.size() * sizeof(uint32_t);
    st = zero::check_hip(hipMalloc(&tab->mem, table_bytes + index_bytes), "zero_muon_table_create: hipMalloc");
    if (st != ZERO_OK) return st;
    char* const at = static_cast<char*>(tab->mem);
    tab->m.table = reinterpret_cast<const Desc*>(at);
    for (int g = 0; g < kGrids; ++g) tab->m.index[g] = reinterpret_cast<const uint32_t*>(at + table_bytes) + starts[g];
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
            d.rows = static_cast<int32_t>(rows[i]);
            d.cols = static_cast<int32_t>(cols[i]);
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
            return int64_t(a.rows) + a.cols > int64_t(b.rows) + b.cols;
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
    }
    c.times = table->times;
    Matrices m = table->m;
    place(&m, workspace, table->partials);
    return launch(m, c, stream, who);
}
