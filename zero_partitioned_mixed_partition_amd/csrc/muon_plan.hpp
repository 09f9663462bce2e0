// What an orthogonalisation by Newton-Schulz steps computes, as a list of
// matrix products, and where its matrices lie in the workspace (host C++, no
// device code).
//
// G is a matrix of m x n, m <= n (a tall matrix is taken transposed). With
// X = G / (|G| + eps) and per step (a, b, c)
//   A = X X^T,   C = a I + b A + c A^2,   X <- C X,
// every A and C is a polynomial of the first A, so they commute and are
// symmetric: products of two of them are computed on the tiles at and below
// the diagonal and mirrored. Two steps can share one pass over X:
//   A' = C A C (the next step's A),   X <- (C' C) X,
// which takes three m^3 products more and one m^2 n product with its X X^T less.
// C' C is symmetric but for the roundings of C, which a mirrored half would let
// grow: where strong directions have converged (a pair after the first) all of
// it is computed.
//
// In flops, r = n / m: a step alone 3 r + 1 times m^3 (A r, its square 1, the
// apply 2 r), the first pair 3 r + 5 against 6 r + 2, another 3 r + 6. Five steps
// in pairs 9 r + 12, with one pair only 12 r + 8, one by one 15 r + 5.
#pragma once

#include <cstdint>
#include <vector>

#include "internal.hpp"

namespace zero {
namespace muon {

// A matrix's arrays in the workspace, all fp16, both sides padded with zeros to multiples of 64 that hold a tile (M >= m,
// N >= n).
enum Buffer : int32_t {
    kX = 0,      // [M][N]: X
    kT0 = 1,     // [N][M]: X transposed, and
    kT1 = 2,     // [N][M]: the one being written while the other is read
    kS0 = 3,     // [M][M]: three square ones for A, C and their products
    kS1 = 4,
    kS2 = 5,
    kLow = 6,    // what rounding X to fp16 left, the source transposed
    kNone = 7,
};

enum class Kind : int32_t {
    kGram,      // square output, the sum runs over N
    kSquare,    // square output, the sum runs over M
    kApply,     // X and its transpose, the sum runs over M
    kFinal,     // as kApply, into the caller's array
};

// out = alpha * kappa^kappa_power * lhs rhs^T + beta * add + diag * I, where an
// apply's rhs is a transposed X. Values are held scaled by powers of two, so
// that fp16 keeps its 11 bits from the largest to 2^-27 of it; the factors hold
// the differences.
struct Product {
    Kind kind;
    int32_t lhs, rhs, add, out, out_t;
    int32_t kappa_power;
    float alpha, beta, diag;
    int32_t low_in;          // an apply: lhs's diagonal times what rounding X left is added to the product
    int32_t low_out;         // and what rounding its own result leaves is kept
    int32_t full;            // a square product: every tile is computed, none mirrored
};

// The most steps one call takes.
constexpr int kMaxSteps = 32;

// The products of n_steps steps. `pairs`: steps in pairs, else one pair and single steps. `low`: the first X has a
// low part. ZERO_EINVAL for steps that let the largest singular value grow past 2^20. Throws std::bad_alloc.
zero_status make_program(const double* coefficients, int32_t n_steps, bool pairs, bool low, std::vector<Product>* out,
                         const char* who);

// ZERO_EINVAL for NULL or non-finite coefficients, or n_steps outside [1, kMaxSteps].
zero_status check_coefficients(const double* coefficients, int32_t n_steps, const char* who);

// Estimated microseconds of a call's products of each kind: X X^T, other square ones, applies.
struct Times {
    double gram, square, apply;
};

// And of its program, for choosing between the two.
double program_time(const Times& t, int32_t n_steps, bool pairs);

// ------------------------------------------------------------ sizes

constexpr int64_t kMaxShort = int64_t(1) << 16;    // the longer and the shorter side at most
constexpr int64_t kMaxLong = int64_t(1) << 22;

// Elements of one workgroup of the momentum pass, and at most so many workgroups (partial sums) a matrix.
constexpr int64_t kChunk = 8192;
constexpr int64_t kMaxChunks = 1024;

// One matrix as the kernels see it. Device tables hold an array of these.
struct alignas(128) Desc {
    const void* src;          // the gradient (bf16), or the orthogonalisation's input
    float* momentum;          // NULL for an orthogonalisation
    float* master;
    uint16_t* out;            // parameters, or the orthogonalised matrix
    int64_t ws;               // byte offset of its arrays in the workspace
    int64_t chunk;            // elements of one workgroup of the momentum pass
    double scale;             // of its update
    int32_t rows, cols;       // the caller's
    int32_t M, N;             // the padded short and long side
    int32_t first_partial;    // its first partial sum
    int32_t chunks;
    int32_t first[5];         // its first workgroup of each grid
    int32_t id;
    int32_t parts;            // workgroups that share its sums over the long side, where the short side is at most 128
    int64_t short_ws;         // byte offset of what they use
};
static_assert(sizeof(Desc) == 128, "one 128-byte descriptor per matrix");

// The grids: by chunk of elements (the momentum pass), by kPack x kPack tile (the packing), by product tile of X (an
// apply), by product tile of a square matrix's lower triangle, and by part of the long side.
enum Grid : int32_t { kByChunk = 0, kByPack = 1, kByTile = 2, kByPair = 3, kByPart = 4 };
constexpr int kGrids = 5;
constexpr int64_t kPack = 64;

constexpr uint32_t kUnits = 256;                 // compute units of the chip

// Values from one row of K to the next: an odd number of 256-byte lines, so that the rows of a tile, which are read at the
// same K, lie in all memory channels (these change every 256 bytes; a power of two of them puts every row in one).
constexpr int32_t stride(int32_t k) { return ((k + 127) / 128 | 1) * 128; }

inline int64_t pad(int64_t x, int64_t tile) { return (x + tile - 1) / tile * tile; }

// The tiles of a call's products by an estimate of five steps' time with each pair: 64, 128, 192 or 256 for those of
// square matrices, 64, 128 or 256 for those with X's shape. Sums over K are measured in stages of 64. Larger tiles read
// less for each product; smaller ones fill the chip from fewer matrices and pad less. 192 is for the last round of
// workgroups, which with 256 can leave half of the chip idle: X X^T of a side of 4096 has 136 tiles of 256 (87 us at K
// 4096) and 253 of 192 (70 us); where both fill whole rounds 256 is up to a sixth faster.
constexpr int kTileSizes = 4;
class TileChoice {
public:
    void add(int64_t count, int64_t rows, int64_t cols);
    void best(int64_t* square, int64_t* rect, Times* times) const;

private:
    struct Total {
        double square = 0, rect = 0;             // tiles
        double gram = 0, squares = 0, apply = 0; // tiles times stages
    } total_[kTileSizes][kTileSizes];
};

// Of `tiles` 256-tiles of square products those that are computed whole: all but a last round that fills at most a
// quarter of the chip, whose quarters then do.
constexpr uint32_t whole_tiles(uint32_t tiles) {
    const uint32_t last = tiles % kUnits;
    return tiles > kUnits && last <= kUnits / 4 ? tiles - last : tiles;
}

// Fills in M, N, chunk and chunks of a matrix of rows x cols, whose sides are padded to `tile` at least.
void shape(Desc* d, int64_t rows, int64_t cols, int64_t tile);

// Workgroups of a matrix in each grid.
int64_t grid_count(const Desc& d, int grid, int64_t square_tile, int64_t rect_tile);

// Bytes of a matrix's arrays.
int64_t area_bytes(const Desc& d);

// ------------------------------------------------------------ matrices with a short side of at most 128
//
// A = X X^T of such a matrix fits a compute unit's LDS. All steps are then taken on A alone, as one group, in two fp16
// parts a value (22 bits), and X is read twice: for A, and for the last product with Q = C_n ... C_1.

// 64, 96 or 128 for a short side up to that, else 0.
inline int32_t short_side(int64_t m) { return m <= 64 ? 64 : m <= 96 ? 96 : m <= 128 ? 128 : 0; }

// One step's factors: C = a + b A + c A^2, then T, the next A and Q from products of what is held.
struct ShortStep {
    float a, b, c, t, next, q;
};
struct ShortProgram {
    int32_t n_steps;
    double first;             // what A is held times
    float last;               // the result is Q X times this
    ShortStep step[kMaxSteps];
};

// Whether the steps can be taken as one group: what rounding A leaves in a direction that the matrix does not have grows
// with the square of each step's a, and must stay well below 1.
bool make_short_program(const double* coefficients, int32_t n_steps, ShortProgram* out);

// Parts of a matrix whose longer side is n, one of `count`: as many as make the sums' two halves (a part's run along
// the long side, and one workgroup's sum over the parts) take equally long, within a chip's worth of workgroups.
int32_t short_parts(int32_t side, int64_t n, int64_t count);

// Bytes of a matrix's Q and parts (with side 128 two more Qs, which a step reads and writes).
constexpr int64_t short_area_bytes(int32_t side, int64_t parts) {
    return 4 * int64_t(side) * side * (parts + (side == 128 ? 3 : 1));
}

// Bytes at the start of the workspace: the parts' exponents, and an exponent and factor per matrix.
inline int64_t short_scales_at(int64_t parts) { return (4 * parts + 7) / 8 * 8; }
inline int64_t short_head_bytes(int64_t parts, int64_t matrices) {
    return (short_scales_at(parts) + 8 * matrices + 255) / 256 * 256;
}

// Bytes at the workspace's start: the partial sums and a factor per matrix.
int64_t head_bytes(int64_t partials, int64_t matrices);

}  // namespace muon
}  // namespace zero
