// AdamW with the two moments held in 8 bits (gfx950): the flat shard, many
// tensors through a device table, and the reduce and the update in one pass;
// and the moments' conversions to and from fp32. The format is state8.hpp's.
//
// "Zero Redundancy Optimizer (ZeRO) and Fully Sharded Data Parallelism (FSDP):
// Mathematical Foundations ...", section "Static Memory Allocation" (fp32
// master, m_t and v_t are 12 of the 16 bytes of a parameter; here the moments
// take 2.02 bytes instead of 8) and "Execution Flow for ZeRO-1" steps 3-4.
//
// Per element: the moments are decoded, updated with the 32-bit AdamW's fp32
// operations in its order (the update uses the fp32 m and v, before they are
// rounded), and encoded with the block's new scale. A block is held by 32
// neighbouring lanes of one wave, so its maximum is a few cross-lane operations
// and every array is read and written once: 16 bytes an element and 4 per block
// of 128.
//
// Bound: HBM. With the moments at a byte, the bytes fall from 28 to 16 while the
// arithmetic grows, to 79 vector instructions an element by the counters (some 45
// issue slots of them the IEEE square root and two divisions), where the memory
// time leaves room for about 97; the conversions in one instruction each are
// what keeps the sum under it. (A square root and reciprocal of 1 ulp in their
// place gain nothing: 348-350 us against 340-351 at 2^27 elements.) The loads are
// not all in flight together: the guards of a last short chunk make the compiler
// wait for a wave's state before it loads the gradient, and for the gradient
// before the clip coefficient. A full chip covers that; small calls pay for each
// (250 k elements: 4.2 us in a graph). Four elements a lane: with 8 a lane's
// two 16-byte stores of the master leave half-written lines behind each other
// and the write-through stores fell to 3.1 TB/s (662 us at 125 M elements); with
// 2 the random words, shared by 8 elements, are computed four times over (about
// 400 us). Measured: 125 M elements 312 us, 6.45 TB/s (a 1 GB copy: 6.55).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <string>
#include <vector>

#include "device_common.hpp"
#include "internal.hpp"
#include "schedule_device.hpp"
#include "state8.hpp"

#pragma clang fp contract(off)

namespace {

using zero::dev::f32x4;
using zero::dev::u32x2;
using zero::dev::u32x4;
using zero::adam::AdamState;
using AdamScalars = zero::adam::StepScalars;
using zero::state8::Words;
using zero::state8::kBlock;

// Two waves a workgroup, four elements a lane. Measured on MI355X, 125 M
// elements: 64 threads 328 us, 128 312 us, 256 318 us, 512 338 us.
constexpr int kThreads = 128;

constexpr int kEpt = zero::state8::kLaneElems;
constexpr int64_t kChunk = int64_t(kThreads) * kEpt;
static_assert(kChunk % kBlock == 0, "whole blocks a workgroup");

// The arrays of one update.
struct Arrays {
    float* p;
    uint8_t* m;
    uint8_t* ms;
    uint8_t* v;
    uint8_t* vs;
    const uint16_t* g;
    uint16_t* o;
};

// One element, in zero_shard_adamw_step's documented order; every line is one
// IEEE fp32 operation.
__device__ __forceinline__ void adam_elem(float& p, float& m, float& v, float g, const AdamScalars& c) {
    const float bm = c.beta1 * m;
    const float gm = c.one_minus_beta1 * g;
    m = bm + gm;
    const float bv = c.beta2 * v;
    const float gg = g * g;
    const float gv = c.one_minus_beta2 * gg;
    v = bv + gv;
    p = p * c.decay;
    const float root = sqrtf(v);
    const float denom = root / c.sqrt_bc2 + c.eps;
    const float ratio = m / denom;
    p = p - c.step_size * ratio;
}

__device__ __forceinline__ float read_clip(const float* clip_scale) {
    return clip_scale != nullptr ? *clip_scale : 1.0f;
}

// The arrays from element `base` (a multiple of the block) on.
__device__ __forceinline__ Arrays from(const Arrays& a, int64_t base) {
    return Arrays{a.p + base, a.m + base, a.ms + base / kBlock, a.v + base, a.vs + base / kBlock, a.g + base, a.o + base};
}

// Elements of a workgroup's chunk at `base` that lie below n, and of a lane's
// kEpt elements from t on.
__device__ __forceinline__ int chunk_left(int64_t n, int64_t base) {
    const int64_t left = n - base;
    return left <= 0 ? 0 : (left < kChunk ? static_cast<int>(left) : static_cast<int>(kChunk));
}
__device__ __forceinline__ int lane_live(int left, uint32_t t) {
    const int live = left - static_cast<int>(t);
    return live <= 0 ? 0 : (live < kEpt ? live : kEpt);
}

// What a lane holds of its elements: those at or past n are zeros.
struct Lane {
    float p[kEpt] = {};
    uint32_t m = 0, v = 0;                 // codes, the first lowest
    uint32_t ms = 0, vs = 0;
    int live = 0;                          // elements below n
};

// A lane's accesses of four elements. VEC: every array is aligned to them, and
// stores write through. Otherwise the same widths at any alignment (the types
// claim none beyond the element's, and the hardware takes them), with
// non-temporal stores, whose lines the L2 completes. Measured on MI355X, 125 M
// elements: 427 us with every array one element off (312 aligned), and 740
// element by element.
template <typename T> struct Four;         // the four elements of an access
template <> struct Four<float> { typedef f32x4 type; };
template <> struct Four<uint16_t> { typedef u32x2 type; };
template <> struct Four<uint8_t> { typedef uint32_t type; };
__device__ __forceinline__ f32x4 load_any(const float* p) {
    typedef f32x4 any __attribute__((aligned(4)));
    return __builtin_nontemporal_load(reinterpret_cast<const any*>(p));
}
__device__ __forceinline__ u32x2 load_any(const uint16_t* p) {
    typedef u32x2 any __attribute__((aligned(2)));
    return __builtin_nontemporal_load(reinterpret_cast<const any*>(p));
}
__device__ __forceinline__ uint32_t load_any(const uint8_t* p) {
    typedef uint32_t any __attribute__((aligned(1)));
    return __builtin_nontemporal_load(reinterpret_cast<const any*>(p));
}
__device__ __forceinline__ void store_any(float* p, f32x4 v) {
    typedef f32x4 any __attribute__((aligned(4)));
    __builtin_nontemporal_store(v, reinterpret_cast<any*>(p));
}
__device__ __forceinline__ void store_any(uint16_t* p, u32x2 v) {
    typedef u32x2 any __attribute__((aligned(2)));
    __builtin_nontemporal_store(v, reinterpret_cast<any*>(p));
}
__device__ __forceinline__ void store_any(uint8_t* p, uint32_t v) {
    typedef uint32_t any __attribute__((aligned(1)));
    __builtin_nontemporal_store(v, reinterpret_cast<any*>(p));
}
template <bool VEC, typename T>
__device__ __forceinline__ typename Four<T>::type load4(const T* p) {
    if (VEC) return zero::dev::ld_stream(reinterpret_cast<const typename Four<T>::type*>(p));
    return load_any(p);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store4(T* base, uint32_t t, const typename Four<T>::type& v) {
    if (VEC)
        zero::dev::st_stream_at(base, sizeof(T) * t, v);
    else
        store_any(base + t, v);
}

// In everything below, the arrays start at the workgroup's chunk (the same
// pointers in every lane) and t is the lane's first element in it, so that a
// wave addresses an array by a scalar base and a 32-bit offset. Lanes with
// fewer than kEpt elements left go one by one.
template <bool VEC>
__device__ __forceinline__ void load_state(Lane& l, const Arrays& a, uint32_t t) {
    if (l.live == kEpt) {
        const f32x4 x = load4<VEC>(a.p + t);
        l.m = load4<VEC>(a.m + t);
        l.v = load4<VEC>(a.v + t);
#pragma unroll
        for (int k = 0; k < kEpt; ++k) l.p[k] = x[k];
    } else {
#pragma unroll
        for (int k = 0; k < kEpt; ++k) {
            if (k < l.live) {
                l.p[k] = a.p[t + k];
                l.m |= static_cast<uint32_t>(a.m[t + k]) << (8 * k);
                l.v |= static_cast<uint32_t>(a.v[t + k]) << (8 * k);
            }
        }
    }
    if (l.live > 0) {
        l.ms = a.ms[t / kBlock];
        l.vs = a.vs[t / kBlock];
    }
}

template <bool VEC>
__device__ __forceinline__ void load_grad(float (&g)[kEpt], const uint16_t* grad, int live, uint32_t t) {
#pragma unroll
    for (int k = 0; k < kEpt; ++k) g[k] = 0.0f;
    if (live == kEpt) {
        const u32x2 x = load4<VEC>(grad + t);
        g[0] = zero::dev::lo_bf16(x[0]);
        g[1] = zero::dev::hi_bf16(x[0]);
        g[2] = zero::dev::lo_bf16(x[1]);
        g[3] = zero::dev::hi_bf16(x[1]);
    } else {
#pragma unroll
        for (int k = 0; k < kEpt; ++k)
            if (k < live) g[k] = zero::dev::bf16_to_f32(grad[t + k]);
    }
}

// Updates a lane's elements from their clipped gradients and writes them back;
// `first` is the number of the chunk's first element, `base` the step's part of
// the random words' keys. Every lane of the wave calls it (the block maxima cross
// lanes); a lane past n brings zeros, which change no maximum.
template <bool VEC>
__device__ __forceinline__ void update_and_store(Lane& l, const float (&g)[kEpt], const Arrays& a, uint32_t t,
                                                 int64_t first, const AdamScalars& c, uint64_t base) {
    float m[kEpt], v[kEpt];
    zero::state8::decode4(l.m, l.ms, m);
    zero::state8::decode4(l.v, l.vs, v);
#pragma unroll
    for (int k = 0; k < kEpt; ++k) adam_elem(l.p[k], m[k], v[k], g[k], c);
    const uint32_t ms = zero::state8::scale_byte(zero::state8::block_max(zero::state8::max_bits4(m)));
    const uint32_t vs = zero::state8::scale_byte(zero::state8::block_max(zero::state8::max_bits4(v)));
    if (l.live == 0) return;
    const Words words = zero::state8::words_at(zero::dev::first_lane(first), t, kChunk, base);
    uint32_t rm[kEpt], rv[kEpt];
    rm[0] = words.a + ((t & 4u) != 0 ? words.b << 2 : 0u);
#pragma unroll
    for (int k = 1; k < kEpt; ++k) rm[k] = rm[k - 1] + words.b;
#pragma unroll
    for (int k = 0; k < kEpt; ++k) rv[k] = rm[k] << 12;      // the word's low 20 bits, as a seed's high ones
    const uint32_t mw = zero::state8::encode4(m, ms, rm);
    const uint32_t vw = zero::state8::positive4(zero::state8::encode4(v, vs, rv), v, vs);
    if (t % kBlock == 0) {                 // the block's first lane
        a.ms[t / kBlock] = static_cast<uint8_t>(ms);
        a.vs[t / kBlock] = static_cast<uint8_t>(vs);
    }
    if (l.live == kEpt) {
        store4<VEC>(a.p, t, f32x4{l.p[0], l.p[1], l.p[2], l.p[3]});
        store4<VEC>(a.m, t, mw);
        store4<VEC>(a.v, t, vw);
        store4<VEC>(a.o, t, u32x2{zero::dev::pack_bf16(l.p[0], l.p[1]),
                                              zero::dev::pack_bf16(l.p[2], l.p[3])});
    } else {
#pragma unroll
        for (int k = 0; k < kEpt; ++k) {
            if (k < l.live) {
                a.p[t + k] = l.p[k];
                a.m[t + k] = static_cast<uint8_t>(mw >> (8 * k));
                a.v[t + k] = static_cast<uint8_t>(vw >> (8 * k));
                a.o[t + k] = static_cast<uint16_t>(zero::dev::f32_to_bf16(l.p[k]));
            }
        }
    }
}

// One workgroup's kChunk elements from `base` of arrays of n elements.
template <bool VEC>
__device__ __forceinline__ void update_chunk(const Arrays& whole, int64_t n, int64_t base, int64_t first,
                                             const AdamScalars& c, uint64_t words, const float* clip_scale) {
    const Arrays a = from(whole, base);
    const uint32_t t = threadIdx.x * kEpt;
    Lane l;
    l.live = lane_live(chunk_left(n, base), t);
    load_state<VEC>(l, a, t);
    float g[kEpt];
    load_grad<VEC>(g, a.g, l.live, t);
    const float clip = read_clip(clip_scale);   // last: the compiler waits for the gradient first
    if (!isfinite(clip)) return;                // the same in every lane
#pragma unroll
    for (int k = 0; k < kEpt; ++k) g[k] = g[k] * clip;
    update_and_store<VEC>(l, g, a, t, first + base, c, words);
}

// The step's scalars and its part of the random words' keys: from the call, or
// from a schedule's state.
struct CallStep {
    AdamScalars c;
    uint64_t base;
    __device__ __forceinline__ AdamScalars scalars() const { return c; }
    __device__ __forceinline__ uint64_t words() const { return base; }
};
struct ScheduleStep {
    const AdamState* state;
    uint64_t seed;
    __device__ __forceinline__ AdamScalars scalars() const { return state->next; }
    __device__ __forceinline__ uint64_t words() const {
        return zero::state8::step_base(seed, static_cast<uint64_t>(state->applied + 1));
    }
};

__device__ __forceinline__ int64_t workgroup() {
    return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

template <bool VEC, typename Step>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(Arrays a, int64_t n, int64_t first, Step step,
                                                          const float* __restrict__ clip_scale) {
    update_chunk<VEC>(a, n, workgroup() * kChunk, first, step.scalars(), step.words(), clip_scale);
}

// Many tensors: one 128-byte descriptor per non-empty tensor and, per
// workgroup, the index of its descriptor. Pointers read from memory have no
// address space, so this kernel's loads are flat instructions with 64-bit
// addresses in the lanes (81-83 vector instructions an element; 148 tensors of
// 15.6 M elements 44 us, the flat shard of as many 42.8).
struct alignas(128) Desc {
    Arrays a;
    int64_t n;
    int64_t first;          // the tensor's first element, in the list's numbering of random words
    int64_t first_block;
    int64_t vec;
};
static_assert(sizeof(Desc) == 128, "one 128-byte descriptor per tensor");

template <typename Step>
__global__ __launch_bounds__(kThreads) void adamw8_table_kernel(const Desc* __restrict__ table,
                                                                const uint32_t* __restrict__ index,
                                                                int64_t blk0, int64_t per, Step step,
                                                                const float* __restrict__ clip_scale) {
    const int64_t blk = blk0 + static_cast<int64_t>(blockIdx.x);
    const Desc d = table[index[zero::dev::xcd_major_entry(blk0, per)]];
    const int64_t base = (blk - d.first_block) * kChunk;
    if (d.vec)
        update_chunk<true>(d.a, d.n, base, d.first, step.scalars(), step.words(), clip_scale);
    else
        update_chunk<false>(d.a, d.n, base, d.first, step.scalars(), step.words(), clip_scale);
}

// The list form, for buffers that move from step to step: the descriptors
// travel in the kernel arguments, and a workgroup finds its tensor by a binary
// search over the tensors' first workgroups.
constexpr int kListTensors = 48;
struct ListBatch {
    Arrays a[kListTensors];
    int64_t n[kListTensors];
    int64_t first[kListTensors];
    int32_t first_block[kListTensors + 1];
    int32_t count;
    uint64_t vec;                          // bit k: tensor k takes vector accesses
};
static_assert(sizeof(ListBatch) + sizeof(CallStep) + sizeof(float*) <= 4096, "kernel arguments are limited to 4 KB");

__global__ __launch_bounds__(kThreads) void adamw8_list_kernel(ListBatch b, CallStep step,
                                                               const float* __restrict__ clip_scale) {
    const int32_t blk = static_cast<int32_t>(blockIdx.x);
    int lo = 0, hi = b.count - 1;          // k with first_block[k] <= blk < first_block[k + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first_block[mid] <= blk) lo = mid; else hi = mid - 1;
    }
    const int64_t base = static_cast<int64_t>(blk - b.first_block[lo]) * kChunk;
    if ((b.vec >> lo) & 1u)
        update_chunk<true>(b.a[lo], b.n[lo], base, b.first[lo], step.c, step.base, clip_scale);
    else
        update_chunk<false>(b.a[lo], b.n[lo], base, b.first[lo], step.c, step.base, clip_scale);
}

// The reduce and the update in one pass: the averaged gradient is the
// reduce's (fp32 sum in replica order, one division by R, one rounding to
// bf16), used where it is formed.
struct Replicas {
    const uint16_t* p[ZERO_MAX_REPLICAS];
};
// Replica loads in flight per lane (B). A full chip has waves enough to cover
// the latency of two at a time, and keeps its streams in order: 164 M elements
// of 8 replicas take 781 us with B = 2, 786 with 3, 809 with 4 or 8; 32 M of 64
// replicas 745, 787 and 805. A window that the chip holds at once waits for
// each load: 1 M elements of 8 replicas take 8.2 us with B = 2 and 7.0 with 8,
// of 64 replicas 29.3 and 24.6 (4 M of 8: 22.5 and 21.3; 8 M: 42.8 and 42.6). A
// batch of 8 loads its first replica again in place of each that it lacks, so
// few replicas take B = 2 (120 M of 2: 354 us against 422).
constexpr int kWideBatch = 8, kBatch = 2;
inline bool wide_batch(int64_t n, int32_t n_replicas) {
    return n <= (int64_t(1) << 22) && n_replicas > kWideBatch / 2;
}

template <bool VEC, int B>
__device__ __forceinline__ void mean_grad(float (&g)[kEpt], const Replicas& reps, int n_rep, int64_t src_off,
                                          int live, uint32_t t) {
    float acc[kEpt] = {};
    if (live == kEpt) {
        const auto add = [&](u32x2 x) {
            acc[0] = acc[0] + zero::dev::lo_bf16(x[0]);
            acc[1] = acc[1] + zero::dev::hi_bf16(x[0]);
            acc[2] = acc[2] + zero::dev::lo_bf16(x[1]);
            acc[3] = acc[3] + zero::dev::hi_bf16(x[1]);
        };
        if (VEC) {
            zero::dev::for_replicas<B, u32x2>(reps.p, n_rep, src_off, t / kEpt, add);
        } else {
            for (int r = 0; r < n_rep; ++r) add(load4<false>(reps.p[r] + src_off + t));
        }
    } else if (live > 0) {
        for (int r = 0; r < n_rep; ++r) {
            const uint16_t* p = reps.p[r] + src_off;
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < live) acc[k] = acc[k] + zero::dev::bf16_to_f32(p[t + k]);
        }
    }
    const float count = static_cast<float>(n_rep);
#pragma unroll
    for (int k = 0; k < kEpt; ++k)
        g[k] = zero::dev::bf16_to_f32(zero::dev::f32_to_bf16(acc[k] / count));
}

template <bool VEC, int B, typename Step>
__global__ __launch_bounds__(kThreads) void reduce_adamw8_kernel(Replicas reps, int n_rep, int64_t src_off,
                                                                 Arrays whole, uint16_t* __restrict__ grad_out,
                                                                 int64_t n, int64_t first, Step step,
                                                                 const float* __restrict__ clip_scale) {
    const int64_t base = workgroup() * kChunk;
    const Arrays a = from(whole, base);
    const uint32_t t = threadIdx.x * kEpt;
    Lane l;
    l.live = lane_live(chunk_left(n, base), t);
    load_state<VEC>(l, a, t);
    float g[kEpt];
    mean_grad<VEC, B>(g, reps, n_rep, src_off + base, l.live, t);
    if (grad_out != nullptr) {
        uint16_t* const out = grad_out + base;
        if (l.live == kEpt) {
            store4<VEC>(out, t, u32x2{zero::dev::pack_bf16(g[0], g[1]), zero::dev::pack_bf16(g[2], g[3])});
        } else {
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < l.live) out[t + k] = static_cast<uint16_t>(zero::dev::f32_to_bf16(g[k]));
        }
    }
    const float clip = read_clip(clip_scale);
    if (!isfinite(clip)) return;
#pragma unroll
    for (int k = 0; k < kEpt; ++k) g[k] = g[k] * clip;
    update_and_store<VEC>(l, g, a, t, first + base, step.scalars(), step.words());
}

// ------------------------------------------------------------ conversions

// A workgroup converts several chunks (rows), loaded before the first is converted.
// (In dequantize the compiler waits for the first row's scale byte before it loads
// the codes.)
// Measured on MI355X at 125 M elements: quantize with 1, 2, 3, 4, 8 rows 108,
// 98, 102, 102, 105 us; dequantize 138, 116, 104, 103, 113 us.
constexpr int kQuantizeRows = 2, kDequantizeRows = 4;

// fp32 to codes and scales, rounded to nearest even.
template <bool VEC>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const float* __restrict__ x, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, int64_t n, int second) {
    const int64_t base = workgroup() * (kQuantizeRows * kChunk);
    const uint32_t t = threadIdx.x * kEpt;
    float v[kQuantizeRows][kEpt] = {};
    int live[kQuantizeRows];
#pragma unroll
    for (int r = 0; r < kQuantizeRows; ++r) {
        const float* const from_x = x + base + r * kChunk;
        live[r] = lane_live(chunk_left(n, base + r * kChunk), t);
        if (live[r] == kEpt) {
            const f32x4 q = load4<VEC>(from_x + t);
#pragma unroll
            for (int k = 0; k < kEpt; ++k) v[r][k] = q[k];
        } else {
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < live[r]) v[r][k] = from_x[t + k];
        }
    }
#pragma unroll
    for (int r = 0; r < kQuantizeRows; ++r) {
        const uint32_t byte = zero::state8::scale_byte(zero::state8::block_max(zero::state8::max_bits4(v[r])));
        if (live[r] == 0) continue;
        uint32_t w = zero::state8::nearest4(v[r], byte);
        if (second) w = zero::state8::positive4(w, v[r], byte);
        uint8_t* const to = codes + base + r * kChunk;
        if (t % kBlock == 0) scales[(base + r * kChunk) / kBlock + t / kBlock] = static_cast<uint8_t>(byte);
        if (live[r] == kEpt) {
            store4<VEC>(to, t, w);
        } else {
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < live[r]) to[t + k] = static_cast<uint8_t>(w >> (8 * k));
        }
    }
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              float* __restrict__ out, int64_t n) {
    const int64_t base = workgroup() * (kDequantizeRows * kChunk);
    const uint32_t t = threadIdx.x * kEpt;
    uint32_t w[kDequantizeRows] = {}, byte[kDequantizeRows] = {};
    int live[kDequantizeRows];
#pragma unroll
    for (int r = 0; r < kDequantizeRows; ++r) {
        const uint8_t* const from_c = codes + base + r * kChunk;
        live[r] = lane_live(chunk_left(n, base + r * kChunk), t);
        if (live[r] > 0) byte[r] = scales[(base + r * kChunk) / kBlock + t / kBlock];
        if (live[r] == kEpt) {
            w[r] = load4<VEC>(from_c + t);
        } else {
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < live[r]) w[r] |= static_cast<uint32_t>(from_c[t + k]) << (8 * k);
        }
    }
#pragma unroll
    for (int r = 0; r < kDequantizeRows; ++r) {
        if (live[r] == 0) continue;
        float v[kEpt];
        zero::state8::decode4(w[r], byte[r], v);
        float* const to = out + base + r * kChunk;
        if (live[r] == kEpt) {
            store4<VEC>(to, t, f32x4{v[0], v[1], v[2], v[3]});
        } else {
#pragma unroll
            for (int k = 0; k < kEpt; ++k)
                if (k < live[r]) to[t + k] = v[k];
        }
    }
}

// ------------------------------------------------------------ host side

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool vector_ok(const Arrays& a) {
    return aligned(a.p, 16) && aligned(a.m, kEpt) && aligned(a.v, kEpt) && aligned(a.g, 2 * kEpt) &&
           aligned(a.o, 2 * kEpt);
}

// The grid of one array's call: rows of workgroups, since a grid dimension holds
// fewer than 2^32 work-items. At most 2^48 elements, whose rows and bytes fit.
constexpr int64_t kMaxElements = int64_t(1) << 48;
zero_status grid_for(int64_t items, int64_t per_workgroup, dim3* grid, const char* who) {
    constexpr int64_t kMaxRow = (int64_t(1) << 32) / kThreads - 1;
    static_assert(kMaxElements / kChunk / kMaxRow < 0xFFFF, "rows of the largest call");
    if (items > kMaxElements) return zero::fail(ZERO_ERANGE, std::string(who) + ": more than 2^48 elements");
    const int64_t blocks = (items - 1) / per_workgroup + 1;
    const int64_t rows = (blocks + kMaxRow - 1) / kMaxRow;
    *grid = dim3(static_cast<unsigned>((blocks + rows - 1) / rows), static_cast<unsigned>(rows));
    return ZERO_OK;
}

// first: a multiple of the block, and first + n an int64.
zero_status check_first(int64_t first, int64_t n, const char* who) {
    if (first < 0 || first % kBlock != 0)
        return zero::fail(ZERO_EINVAL, std::string(who) + ": first_element must be a multiple of " +
                                           std::to_string(kBlock) + ", >= 0");
    if (n > INT64_MAX - first) return zero::fail(ZERO_ERANGE, std::string(who) + ": first_element + n overflows");
    return ZERO_OK;
}

// "<a> overlaps <b>" for a written array of an update over n > 0 elements, or an
// empty string.
std::string array_clash(const Arrays& a, int64_t n) {
    const size_t nb = static_cast<size_t>(zero::state8::blocks_of(n)), b = static_cast<size_t>(n);
    const zero::Span wr[] = {{a.p, 4 * b, "master"},          {a.m, b, "exp_avg"}, {a.ms, nb, "exp_avg_scale"},
                             {a.v, b, "exp_avg_sq"}, {a.vs, nb, "exp_avg_sq_scale"}, {a.o, 2 * b, "param_out"}};
    const zero::Span rd[] = {{a.g, 2 * b, "grad"}};
    return zero::first_overlap(wr, 6, rd, 1);
}

// The step's scalars and key of a call that counts the steps itself.
zero_status call_step(int64_t step, double lr, double beta1, double beta2, double eps, double weight_decay,
                      uint64_t seed, CallStep* out, const char* who) {
    zero_status st = zero::adam::check_hyper(step, lr, beta1, beta2, eps, weight_decay, who);
    if (st != ZERO_OK) return st;
    st = zero::adam::step_scalars(step, lr, beta1, beta2, weight_decay, eps, &out->c, who);
    out->base = zero::state8::step_base(seed, static_cast<uint64_t>(step));
    return st;
}

bool any_null(const Arrays& a) { return !a.p || !a.m || !a.ms || !a.v || !a.vs || !a.g || !a.o; }

template <typename Step>
zero_status launch_flat(const Arrays& a, int64_t n, int64_t first, const Step& step, const float* clip_scale,
                        hipStream_t stream, const char* who) {
    using zero::fail;
    zero_status st = check_first(first, n, who);
    if (st != ZERO_OK) return st;
    if (n == 0) return ZERO_OK;
    if (any_null(a)) return fail(ZERO_EINVAL, std::string(who) + ": NULL array");
    dim3 grid;
    st = grid_for(n, kChunk, &grid, who);
    if (st != ZERO_OK) return st;
    const std::string clash = array_clash(a, n);
    if (!clash.empty()) return fail(ZERO_EINVAL, std::string(who) + ": " + clash);
    if (vector_ok(a))
        hipLaunchKernelGGL((adamw8_kernel<true, Step>), grid, dim3(kThreads), 0, stream, a, n, first, step, clip_scale);
    else
        hipLaunchKernelGGL((adamw8_kernel<false, Step>), grid, dim3(kThreads), 0, stream, a, n, first, step, clip_scale);
    return zero::check_hip(hipGetLastError(), who);
}

}  // namespace

extern "C" zero_status zero_shard_adamw8_step(float* master, uint8_t* exp_avg, uint8_t* exp_avg_scale,
                                              uint8_t* exp_avg_sq, uint8_t* exp_avg_sq_scale, const uint16_t* grad,
                                              uint16_t* param_out, int64_t n, int64_t first_element, int64_t step,
                                              double lr, double beta1, double beta2, double eps, double weight_decay,
                                              uint64_t seed, const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_shard_adamw8_step";
    zero::clear_error();
    if (n < 0) return zero::fail(ZERO_EINVAL, "zero_shard_adamw8_step: n < 0");
    CallStep s{};
    const zero_status st = call_step(step, lr, beta1, beta2, eps, weight_decay, seed, &s, who);
    if (st != ZERO_OK) return st;
    return launch_flat(Arrays{master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, grad, param_out}, n,
                       first_element, s, clip_scale, stream, who);
}

extern "C" zero_status zero_shard_adamw8_step_scheduled(float* master, uint8_t* exp_avg, uint8_t* exp_avg_scale,
                                                        uint8_t* exp_avg_sq, uint8_t* exp_avg_sq_scale,
                                                        const uint16_t* grad, uint16_t* param_out, int64_t n,
                                                        int64_t first_element, const zero_adamw_schedule* schedule,
                                                        uint64_t seed, const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_shard_adamw8_step_scheduled";
    zero::clear_error();
    if (schedule == nullptr) return zero::fail(ZERO_EINVAL, "zero_shard_adamw8_step_scheduled: NULL schedule");
    if (n < 0) return zero::fail(ZERO_EINVAL, "zero_shard_adamw8_step_scheduled: n < 0");
    const zero_status st = zero::adam::check_schedule_device(schedule, who);
    if (st != ZERO_OK) return st;
    return launch_flat(Arrays{master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, grad, param_out}, n,
                       first_element, ScheduleStep{schedule->state, seed}, clip_scale, stream, who);
}

// ------------------------------------------------------------ many tensors

namespace {

// The checks of a list, and one descriptor per non-empty tensor in list order
// (first_block is the caller's to fill). Throws std::bad_alloc.
zero_status describe_list(float* const* masters, uint8_t* const* exp_avgs, uint8_t* const* exp_avg_scales,
                          uint8_t* const* exp_avg_sqs, uint8_t* const* exp_avg_sq_scales,
                          const uint16_t* const* grads, uint16_t* const* params_out, const int64_t* numels,
                          int32_t n_tensors, int64_t first_element, std::vector<Desc>* descs, const char* who) {
    using zero::fail;
    const std::string w(who);
    if (n_tensors < 0) return fail(ZERO_EINVAL, w + ": n_tensors < 0");
    if (n_tensors > 0 && (!masters || !exp_avgs || !exp_avg_scales || !exp_avg_sqs || !exp_avg_sq_scales || !grads ||
                          !params_out || !numels))
        return fail(ZERO_EINVAL, w + ": NULL array of pointers");
    const zero_status st = check_first(first_element, 0, who);
    if (st != ZERO_OK) return st;
    int64_t first = first_element;
    for (int32_t t = 0; t < n_tensors; ++t) {
        const int64_t n = numels[t];
        const std::string of = " of tensor " + std::to_string(t);
        if (n < 0) return fail(ZERO_EINVAL, w + ": numel < 0" + of);
        if (n == 0) continue;
        if ((n - 1) / kChunk + 1 > 0x7FFFFFFF) return fail(ZERO_ERANGE, w + ": more than 2^31 workgroups" + of);
        const int64_t padded = zero::state8::blocks_of(n) * kBlock;
        if (padded > INT64_MAX - first) return fail(ZERO_ERANGE, w + ": first_element + n overflows" + of);
        Desc d{};
        d.a = Arrays{masters[t], exp_avgs[t], exp_avg_scales[t], exp_avg_sqs[t], exp_avg_sq_scales[t], grads[t],
                     params_out[t]};
        if (any_null(d.a)) return fail(ZERO_EINVAL, w + ": NULL array" + of);
        const std::string clash = array_clash(d.a, n);
        if (!clash.empty()) return fail(ZERO_EINVAL, w + ": " + clash + of);
        d.n = n;
        d.first = first;
        d.vec = vector_ok(d.a);
        descs->push_back(d);
        first += padded;
    }
    return ZERO_OK;
}

}  // namespace

extern "C" zero_status zero_multi_tensor_adamw8_step(float* const* masters, uint8_t* const* exp_avgs,
                                                     uint8_t* const* exp_avg_scales, uint8_t* const* exp_avg_sqs,
                                                     uint8_t* const* exp_avg_sq_scales, const uint16_t* const* grads,
                                                     uint16_t* const* params_out, const int64_t* numels,
                                                     int32_t n_tensors, int64_t first_element, int64_t step, double lr,
                                                     double beta1, double beta2, double eps, double weight_decay,
                                                     uint64_t seed, const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_multi_tensor_adamw8_step";
    zero::clear_error();
    CallStep s{};
    zero_status st = call_step(step, lr, beta1, beta2, eps, weight_decay, seed, &s, who);
    if (st != ZERO_OK) return st;
    std::vector<Desc> descs;
    try {
        st = describe_list(masters, exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, grads, params_out, numels,
                           n_tensors, first_element, &descs, who);
        if (st != ZERO_OK) return st;
        // Largest first, as the 32-bit list: the many small tensors then share a launch.
        std::stable_sort(descs.begin(), descs.end(), [](const Desc& x, const Desc& y) { return x.n > y.n; });
    } catch (const std::bad_alloc&) {
        return zero::fail(ZERO_ENOMEM, "zero_multi_tensor_adamw8_step: host allocation failed");
    }
    constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / kThreads - 1;      // fewer than 2^32 work-items a launch
    if (!descs.empty() && (descs[0].n - 1) / kChunk + 1 > kMaxBlocks)
        return zero::fail(ZERO_ERANGE, "zero_multi_tensor_adamw8_step: a tensor too large for one launch");
    for (size_t at = 0; at < descs.size();) {
        ListBatch b{};
        while (at < descs.size() && b.count < kListTensors) {
            const int k = b.count;
            const int64_t end = b.first_block[k] + ((descs[at].n - 1) / kChunk + 1);
            if (end > kMaxBlocks) break;
            b.a[k] = descs[at].a;
            b.n[k] = descs[at].n;
            b.first[k] = descs[at].first;
            b.vec |= static_cast<uint64_t>(descs[at].vec != 0) << k;
            b.first_block[k + 1] = static_cast<int32_t>(end);
            ++b.count;
            ++at;
        }
        hipLaunchKernelGGL(adamw8_list_kernel, dim3(static_cast<unsigned>(b.first_block[b.count])), dim3(kThreads), 0,
                           stream, b, s, clip_scale);
        st = zero::check_hip(hipGetLastError(), who);
        if (st != ZERO_OK) return st;
    }
    return ZERO_OK;
}

struct zero_mt8_table {
    int device = -1;
    void* mem = nullptr;          // descriptors, then the per-workgroup index
    const Desc* table = nullptr;
    const uint32_t* index = nullptr;
    int64_t blocks = 0;           // workgroups of one step
};

extern "C" zero_status zero_mt8_table_create(float* const* masters, uint8_t* const* exp_avgs,
                                             uint8_t* const* exp_avg_scales, uint8_t* const* exp_avg_sqs,
                                             uint8_t* const* exp_avg_sq_scales, const uint16_t* const* grads,
                                             uint16_t* const* params_out, const int64_t* numels, int32_t n_tensors,
                                             int64_t first_element, zero_mt8_table** out) {
    using zero::fail;
    static const char* const who = "zero_mt8_table_create";
    zero::clear_error();
    const std::string w(who);
    if (!out) return fail(ZERO_EINVAL, w + ": NULL out");
    *out = nullptr;
    zero_status st = ZERO_OK;
    std::vector<Desc> descs;
    std::vector<uint32_t> index;
    zero_mt8_table* tab = nullptr;
    try {
        st = describe_list(masters, exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, grads, params_out, numels,
                           n_tensors, first_element, &descs, who);
        if (st != ZERO_OK) return st;
        int64_t blocks = 0;
        for (size_t k = 0; k < descs.size(); ++k) {
            const int64_t wgs = (descs[k].n - 1) / kChunk + 1;
            if (blocks + wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, w + ": more than 2^31 workgroups in one list");
            descs[k].first_block = blocks;
            index.insert(index.end(), static_cast<size_t>(wgs), static_cast<uint32_t>(k));
            blocks += wgs;
        }
        if (blocks > 0) index = zero::xcd_major_index(index);
        tab = new zero_mt8_table;
        tab->blocks = blocks;
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ENOMEM, w + ": host allocation failed");
    }
    if (tab->blocks > 0) {        // an empty list needs no device
        st = zero::check_hip(hipGetDevice(&tab->device), "zero_mt8_table_create: hipGetDevice");
        const size_t table_bytes = descs.size() * sizeof(Desc), index_bytes = index.size() * sizeof(uint32_t);
        if (st == ZERO_OK)
            st = zero::check_hip(hipMalloc(&tab->mem, table_bytes + index_bytes), "zero_mt8_table_create: hipMalloc");
        if (st == ZERO_OK) {
            tab->table = static_cast<const Desc*>(tab->mem);
            tab->index = reinterpret_cast<const uint32_t*>(static_cast<char*>(tab->mem) + table_bytes);
            st = zero::check_hip(hipMemcpy(tab->mem, descs.data(), table_bytes, hipMemcpyHostToDevice),
                                 "zero_mt8_table_create: hipMemcpy");
        }
        if (st == ZERO_OK)
            st = zero::check_hip(hipMemcpy(const_cast<uint32_t*>(tab->index), index.data(), index_bytes,
                                           hipMemcpyHostToDevice), "zero_mt8_table_create: hipMemcpy");
    }
    if (st != ZERO_OK) {
        if (tab->mem) (void)hipFree(tab->mem);
        delete tab;
        return st;
    }
    *out = tab;
    return ZERO_OK;
}

extern "C" void zero_mt8_table_free(zero_mt8_table* table) {
    if (!table) return;
    if (table->mem) (void)hipFree(table->mem);
    delete table;
}

extern "C" int64_t zero_mt8_table_blocks(const zero_mt8_table* table) { return table ? table->blocks : -1; }

namespace {

template <typename Step>
zero_status launch_table(const zero_mt8_table* table, const Step& step, const float* clip_scale, hipStream_t stream,
                         const char* who) {
    // A dispatch holds fewer than 2^32 work-items: longer lists take several launches.
    constexpr int64_t kMaxBlocks = zero::kTableLaunchBlocks;
    for (int64_t b0 = 0; b0 < table->blocks; b0 += kMaxBlocks) {
        const int64_t nb = table->blocks - b0 < kMaxBlocks ? table->blocks - b0 : kMaxBlocks;
        hipLaunchKernelGGL(adamw8_table_kernel<Step>, dim3(static_cast<unsigned>(nb)), dim3(kThreads), 0, stream,
                           table->table, table->index, b0, (nb + 7) / 8, step, clip_scale);
        const zero_status st = zero::check_hip(hipGetLastError(), who);
        if (st != ZERO_OK) return st;
    }
    return ZERO_OK;
}

zero_status check_table_device(const zero_mt8_table* table, const char* who) {
    int dev = -1;
    const zero_status st = zero::check_hip(hipGetDevice(&dev), who);
    if (st != ZERO_OK) return st;
    if (dev != table->device)
        return zero::fail(ZERO_EINVAL, std::string(who) + ": the table lives on device " +
                                           std::to_string(table->device) + ", the current device is " +
                                           std::to_string(dev));
    return ZERO_OK;
}

}  // namespace

extern "C" zero_status zero_mt8_table_adamw8_step(const zero_mt8_table* table, int64_t step, double lr, double beta1,
                                                  double beta2, double eps, double weight_decay, uint64_t seed,
                                                  const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_mt8_table_adamw8_step";
    zero::clear_error();
    if (!table) return zero::fail(ZERO_EINVAL, "zero_mt8_table_adamw8_step: NULL table");
    CallStep s{};
    zero_status st = call_step(step, lr, beta1, beta2, eps, weight_decay, seed, &s, who);
    if (st != ZERO_OK) return st;
    if (table->blocks == 0) return ZERO_OK;
    st = check_table_device(table, who);
    if (st != ZERO_OK) return st;
    return launch_table(table, s, clip_scale, stream, who);
}

extern "C" zero_status zero_mt8_table_adamw8_step_scheduled(const zero_mt8_table* table,
                                                            const zero_adamw_schedule* schedule, uint64_t seed,
                                                            const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_mt8_table_adamw8_step_scheduled";
    zero::clear_error();
    if (!table || !schedule)
        return zero::fail(ZERO_EINVAL, "zero_mt8_table_adamw8_step_scheduled: NULL table or schedule");
    zero_status st = zero::adam::check_schedule_device(schedule, who);
    if (st != ZERO_OK) return st;
    if (table->blocks == 0) return ZERO_OK;
    st = check_table_device(table, who);
    if (st != ZERO_OK) return st;
    return launch_table(table, ScheduleStep{schedule->state, seed}, clip_scale, stream, who);
}

// ------------------------------------------------------------ reduce and update

namespace {

template <typename Step>
zero_status launch_reduce(const zero_plan* plan, int32_t rank, const uint16_t* const* replicas, int32_t n_replicas,
                          int64_t begin, int64_t count, Arrays a, uint16_t* shard_grad, int64_t first,
                          const Step& step, const float* clip_scale, hipStream_t stream, const char* who) {
    using zero::fail;
    const std::string w(who);
    if (plan == nullptr || replicas == nullptr) return fail(ZERO_EINVAL, w + ": NULL plan or replicas");
    if (rank < 0 || rank >= plan->n_ranks) return fail(ZERO_EINVAL, w + ": rank out of range");
    if (n_replicas < 1 || n_replicas > ZERO_MAX_REPLICAS)
        return fail(ZERO_EINVAL, w + ": n_replicas must be 1.." + std::to_string(ZERO_MAX_REPLICAS));
    if (begin < 0 || count < 0 || begin > plan->padded || count > plan->padded - begin)
        return fail(ZERO_EINVAL, w + ": window outside [0, P)");
    zero_status st = check_first(first, plan->shard, who);
    if (st != ZERO_OK) return st;
    const int64_t shard_lo = static_cast<int64_t>(rank) * plan->shard, shard_hi = shard_lo + plan->shard;
    const int64_t lo = std::max(begin, shard_lo), hi = std::min(begin + count, shard_hi);
    if (lo >= hi) return ZERO_OK;
    const int64_t at = lo - shard_lo, n = hi - lo, src_off = lo - begin;
    if (at % kBlock != 0 || (hi != shard_hi && n % kBlock != 0))
        return fail(ZERO_EINVAL, w + ": the window's part of the shard [" + std::to_string(at) + ", " +
                                     std::to_string(at + n) + ") must start and end at multiples of " +
                                     std::to_string(kBlock) + " elements or the shard's end");
    dim3 grid;
    st = grid_for(n, kChunk, &grid, who);
    if (st != ZERO_OK) return st;
    a.g = replicas[0];
    if (any_null(a)) return fail(ZERO_EINVAL, w + (replicas[0] ? ": NULL state array" : ": NULL replica"));
    Replicas table{};
    for (int32_t k = 0; k < n_replicas; ++k) {
        if (replicas[k] == nullptr) return fail(ZERO_EINVAL, w + ": NULL replica");
        table.p[k] = replicas[k];
    }
    a = Arrays{a.p + at, a.m + at, a.ms + at / kBlock, a.v + at, a.vs + at / kBlock, nullptr, a.o + at};
    uint16_t* const grad_out = shard_grad != nullptr ? shard_grad + at : nullptr;
    const size_t b = static_cast<size_t>(n), nb = static_cast<size_t>(zero::state8::blocks_of(n));
    const zero::Span wr[] = {{a.p, 4 * b, "master"},          {a.m, b, "exp_avg"}, {a.ms, nb, "exp_avg_scale"},
                             {a.v, b, "exp_avg_sq"}, {a.vs, nb, "exp_avg_sq_scale"}, {a.o, 2 * b, "param_out"},
                             {grad_out, grad_out ? 2 * b : 0, "shard_grad"}};
    zero::Span rd[ZERO_MAX_REPLICAS];
    for (int32_t k = 0; k < n_replicas; ++k) rd[k] = {replicas[k] + src_off, 2 * b, "replica", k};
    const std::string clash = zero::first_overlap(wr, 7, rd, n_replicas);
    if (!clash.empty()) return fail(ZERO_EINVAL, w + ": " + clash);
    bool vec = vector_ok(a) && (grad_out == nullptr || aligned(grad_out, 2 * kEpt));
    for (int32_t k = 0; k < n_replicas; ++k) vec = vec && aligned(replicas[k] + src_off, 2 * kEpt);
    const auto kernel = !vec ? reduce_adamw8_kernel<false, kBatch, Step>
                             : (wide_batch(n, n_replicas) ? reduce_adamw8_kernel<true, kWideBatch, Step>
                                                          : reduce_adamw8_kernel<true, kBatch, Step>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, table, n_replicas, src_off, a, grad_out, n, first + at,
                       step, clip_scale);
    return zero::check_hip(hipGetLastError(), who);
}

}  // namespace

extern "C" zero_status zero_reduce_adamw8_step(const zero_plan* plan, int32_t rank, const uint16_t* const* replicas,
                                               int32_t n_replicas, int64_t begin, int64_t count, float* master,
                                               uint8_t* exp_avg, uint8_t* exp_avg_scale, uint8_t* exp_avg_sq,
                                               uint8_t* exp_avg_sq_scale, uint16_t* param_out, uint16_t* shard_grad,
                                               int64_t first_element, int64_t step, double lr, double beta1,
                                               double beta2, double eps, double weight_decay, uint64_t seed,
                                               const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_reduce_adamw8_step";
    zero::clear_error();
    CallStep s{};
    const zero_status st = call_step(step, lr, beta1, beta2, eps, weight_decay, seed, &s, who);
    if (st != ZERO_OK) return st;
    return launch_reduce(plan, rank, replicas, n_replicas, begin, count,
                         Arrays{master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, nullptr, param_out},
                         shard_grad, first_element, s, clip_scale, stream, who);
}

extern "C" zero_status zero_reduce_adamw8_step_scheduled(
    const zero_plan* plan, int32_t rank, const uint16_t* const* replicas, int32_t n_replicas, int64_t begin,
    int64_t count, float* master, uint8_t* exp_avg, uint8_t* exp_avg_scale, uint8_t* exp_avg_sq,
    uint8_t* exp_avg_sq_scale, uint16_t* param_out, uint16_t* shard_grad, int64_t first_element,
    const zero_adamw_schedule* schedule, uint64_t seed, const float* clip_scale, hipStream_t stream) {
    static const char* const who = "zero_reduce_adamw8_step_scheduled";
    zero::clear_error();
    if (schedule == nullptr) return zero::fail(ZERO_EINVAL, "zero_reduce_adamw8_step_scheduled: NULL schedule");
    const zero_status st = zero::adam::check_schedule_device(schedule, who);
    if (st != ZERO_OK) return st;
    return launch_reduce(plan, rank, replicas, n_replicas, begin, count,
                         Arrays{master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, nullptr, param_out},
                         shard_grad, first_element, ScheduleStep{schedule->state, seed}, clip_scale, stream, who);
}

// ------------------------------------------------------------ conversions

extern "C" zero_status zero_state8_quantize(const float* x, int64_t n, int32_t second_moment, uint8_t* codes,
                                            uint8_t* scales, hipStream_t stream) {
    using zero::fail;
    static const char* const who = "zero_state8_quantize";
    zero::clear_error();
    if (n < 0) return fail(ZERO_EINVAL, "zero_state8_quantize: n < 0");
    if (n == 0) return ZERO_OK;
    if (!x || !codes || !scales) return fail(ZERO_EINVAL, "zero_state8_quantize: NULL array");
    dim3 grid;
    const zero_status st = grid_for(n, kQuantizeRows * kChunk, &grid, who);
    if (st != ZERO_OK) return st;
    const size_t b = static_cast<size_t>(n);
    const zero::Span wr[] = {{codes, b, "codes"}, {scales, static_cast<size_t>(zero::state8::blocks_of(n)), "scales"}};
    const zero::Span rd[] = {{x, 4 * b, "x"}};
    const std::string clash = zero::first_overlap(wr, 2, rd, 1);
    if (!clash.empty()) return fail(ZERO_EINVAL, "zero_state8_quantize: " + clash);
    if (aligned(x, 16) && aligned(codes, 4))
        hipLaunchKernelGGL(quantize_kernel<true>, grid, dim3(kThreads), 0, stream, x, codes, scales, n, second_moment);
    else
        hipLaunchKernelGGL(quantize_kernel<false>, grid, dim3(kThreads), 0, stream, x, codes, scales, n, second_moment);
    return zero::check_hip(hipGetLastError(), who);
}

extern "C" zero_status zero_state8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, float* out,
                                              hipStream_t stream) {
    using zero::fail;
    static const char* const who = "zero_state8_dequantize";
    zero::clear_error();
    if (n < 0) return fail(ZERO_EINVAL, "zero_state8_dequantize: n < 0");
    if (n == 0) return ZERO_OK;
    if (!codes || !scales || !out) return fail(ZERO_EINVAL, "zero_state8_dequantize: NULL array");
    dim3 grid;
    const zero_status st = grid_for(n, kDequantizeRows * kChunk, &grid, who);
    if (st != ZERO_OK) return st;
    const size_t b = static_cast<size_t>(n);
    const zero::Span wr[] = {{out, 4 * b, "out"}};
    const zero::Span rd[] = {{codes, b, "codes"}, {scales, static_cast<size_t>(zero::state8::blocks_of(n)), "scales"}};
    const std::string clash = zero::first_overlap(wr, 1, rd, 2);
    if (!clash.empty()) return fail(ZERO_EINVAL, "zero_state8_dequantize: " + clash);
    if (aligned(out, 16) && aligned(codes, 4))
        hipLaunchKernelGGL(dequantize_kernel<true>, grid, dim3(kThreads), 0, stream, codes, scales, out, n);
    else
        hipLaunchKernelGGL(dequantize_kernel<false>, grid, dim3(kThreads), 0, stream, codes, scales, out, n);
    return zero::check_hip(hipGetLastError(), who);
}
