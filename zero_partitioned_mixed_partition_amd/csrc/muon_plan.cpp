// The products and the workspace of an orthogonalisation (muon_plan.hpp).
#include "muon_plan.hpp"

#include <algorithm>
#include <cmath>
#include <string>

namespace zero {
namespace muon {

namespace {

// The power of two e for which values up to `bound` are held as value * 2^e: the largest lies in (2^13, 2^14], a
// factor of 4 below fp16's largest for what roundings add.
int exponent_for(double bound) { return 14 - static_cast<int>(std::ceil(std::log2(std::max(std::min(bound, 1e30), 1e-6)))); }

float pow2(int e) { return static_cast<float>(std::ldexp(1.0, e)); }

constexpr int kSamples = 1024;

// The largest |f(x)| over [0, top], by samples.
template <typename F>
double largest(double top, F f) {
    double most = 0.0;
    for (int i = 0; i <= kSamples; ++i) most = std::max(most, std::fabs(f(top * i / kSamples)));
    return most;
}

// For an exponent: a margin for what lies between the samples.
int exponent_for_largest(double most) { return exponent_for(1.02 * most); }

// A step's factor a + b x + c x^2 and what is made of it, with their largest absolute values over [0, top]: at its end or where
// the derivative is 0.
struct Step {
    double a, b, c;

    double at(double x) const { return a + x * (b + x * c); }
    double left(double x) const { return x * at(x) * at(x); }            // the eigenvalue that it leaves of x
    double largest_factor(double top) const {
        const double x = c != 0.0 ? -b / (2.0 * c) : 0.0;
        return std::max({std::fabs(a), std::fabs(at(top)), x > 0.0 && x < top ? std::fabs(at(x)) : 0.0});
    }
    double largest_times_x(double top) const {
        return over(top, 2.0 * b, 3.0 * c, [&](double x) { return std::fabs(x * at(x)); });
    }
    double largest_left(double top) const {
        return over(top, 3.0 * b, 5.0 * c, [&](double x) { return left(x); });
    }

private:
    // The largest f at top and at the roots of a + p x + q x^2 in (0, top).
    template <typename F>
    double over(double top, double p, double q, F f) const {
        double most = f(top);
        const double under = p * p - 4.0 * a * q;
        if (under < 0.0) return most;
        const double h = -0.5 * (p + std::copysign(std::sqrt(under), p));
        for (const double x : {h != 0.0 ? a / h : 0.0, q != 0.0 ? h / q : 0.0})
            if (x > 0.0 && x < top) most = std::max(most, f(x));
        return most;
    }
};

Step step_at(const double* coefficients, int32_t i) { return {coefficients[3 * i], coefficients[3 * i + 1], coefficients[3 * i + 2]}; }

// How far the roundings of a step can carry an eigenvalue of X X^T past the end of its interval, relative to it. An fp16
// value is off by at most 2^-11 of itself, and X counts twice, A once, C twice; in two fp16 parts 2^-22 of it.
constexpr double kSlack = 5.0 / (1 << 11), kShortSlack = 5.0 / (1 << 22);

// Whether every interval that the steps leave stays within a quarter of itself where roundings make each longer.
bool steady(const double* coefficients, int32_t n_steps, double slack) {
    double exact = 1.0, longer = 1.0;
    for (int32_t i = 0; i < n_steps; ++i) {
        exact = step_at(coefficients, i).largest_left(exact);
        longer = step_at(coefficients, i).largest_left(longer * (1.0 + slack));
        if (!(longer <= 1.25 * exact)) return false;
    }
    return true;
}

// Steps that contract to the very end of an interval and grow steeply past it (the published Polar Express coefficients
// end so) are taken of X / kSafety, all but the last: past the end then lies 2.9e-3 of the eigenvalue, more than kSlack.
constexpr double kSafety = 1.0 + 3.0 / (1 << 11);

}  // namespace

zero_status check_coefficients(const double* coefficients, int32_t n_steps, const char* who) {
    const std::string w(who);
    if (n_steps < 1 || n_steps > kMaxSteps)
        return fail(ZERO_EINVAL, w + ": n_steps must be 1.." + std::to_string(kMaxSteps));
    if (!coefficients) return fail(ZERO_EINVAL, w + ": NULL coefficients");
    for (int32_t i = 0; i < 3 * n_steps; ++i)
        if (!std::isfinite(coefficients[i])) return fail(ZERO_EINVAL, w + ": a coefficient is not finite");
    return ZERO_OK;
}

double program_time(const Times& t, int32_t n_steps, bool pairs) {
    const int32_t two = n_steps < 2 ? 0 : pairs ? n_steps / 2 : 1, one = n_steps - 2 * two;
    return two * (t.gram + 5 * t.square + t.apply) + std::max(two - 1, 0) * t.square + one * (t.gram + t.square + t.apply);
}

zero_status make_program(const double* coefficients, int32_t n_steps, bool pairs, bool low, std::vector<Product>* out,
                         const char* who) {
    out->clear();
    double taken[3 * kMaxSteps];
    std::copy(coefficients, coefficients + 3 * n_steps, taken);
    if (!steady(coefficients, n_steps, kSlack)) {
        for (int32_t i = 0; i + 1 < n_steps; ++i) {
            const double s2 = kSafety * kSafety;
            taken[3 * i] /= kSafety;
            taken[3 * i + 1] /= kSafety * s2;
            taken[3 * i + 2] /= kSafety * s2 * s2;
        }
        if (!steady(taken, n_steps, kSlack)) std::copy(coefficients, coefficients + 3 * n_steps, taken);
    }
    int eX = 14;             // the first X: kappa * 2^-14 times what is held
    double top = 1.0 + kSlack;       // bound of the eigenvalues of A, X X^T of a matrix of norm 1, with what roundings add
    int32_t from = kT0, to = kT1;
    bool kept = low;         // whether there is what rounding X left
    for (int32_t at = 0; at < n_steps;) {
        const bool first = at == 0;
        const Step s0 = step_at(taken, at);
        // (in the pair's A' roundings grow by the square of its first step's a)
        const bool pair = at + 1 < n_steps && (pairs || first) && std::fabs(s0.a) <= 4.0;
        auto product = [&](Kind kind, int32_t lhs, int32_t rhs, int32_t o, double alpha) {
            Product p{};
            p.kind = kind;
            p.lhs = lhs, p.rhs = rhs, p.out = o, p.add = kNone, p.out_t = kNone;
            p.alpha = static_cast<float>(alpha);
            out->push_back(p);
            return &out->back();
        };
        auto polynomial = [&](const Step& s, int32_t from_s, int32_t to_s, int eA, int eC) {
            Product* p = product(Kind::kSquare, from_s, from_s, to_s, s.c * pow2(eC - 2 * eA));
            p->add = from_s;
            p->beta = static_cast<float>(s.b * pow2(eC - eA));
            p->diag = static_cast<float>(s.a * pow2(eC));
        };
        // (A factor that large on an interval that the steps before made that small: the exponents would not fit a float.)
        const auto too_large = [](const Step& s, double end) { return !(s.largest_factor(end) <= 0x1p60); };
        const double between = s0.largest_left(top) * (1.0 + kSlack);        // the end of the interval after this step
        if (too_large(s0, top) || (pair && too_large(step_at(taken, at + 1), between)))
            return fail(ZERO_EINVAL, std::string(who) + ": a step with these coefficients multiplies by more than 2^60");
        const int eA = exponent_for_largest(top), eC = exponent_for_largest(s0.largest_factor(top));
        product(Kind::kGram, kX, kX, kS0, pow2(eA - 2 * eX))->kappa_power = first ? 2 : 0;
        polynomial(s0, kS0, kS1, eA, eC);
        int32_t q = kS1;
        int eQ = eC;
        double next = s0.largest_left(top);
        if (pair) {
            const Step s1 = step_at(taken, at + 1);
            const int eT = exponent_for_largest(s0.largest_times_x(top));
            const int eA1 = exponent_for_largest(between), eC1 = exponent_for_largest(s1.largest_factor(between));
            eQ = exponent_for_largest(largest(top, [&](double x) { return s0.at(x) * s1.at(s0.left(x)); }));
            product(Kind::kSquare, kS1, kS0, kS2, pow2(eT - eC - eA));
            product(Kind::kSquare, kS2, kS1, kS0, pow2(eA1 - eT - eC));
            polynomial(s1, kS0, kS2, eA1, eC1);
            // (Emulated, two pairs and a step: 32 directions over a floor of 1e-3 1.0e-2 with it mirrored, 5.3e-3 so; the first
            // pair's as exact either way but for rank 1, 4.2e-3 and 3.6e-3.)
            product(Kind::kSquare, kS2, kS1, kS0, pow2(eQ - eC1 - eC))->full = !first;
            q = kS0;
            next = s1.largest_left(between);
        }
        if (!(next <= std::ldexp(1.0, 40)))
            return fail(ZERO_EINVAL, std::string(who) + ": these coefficients let singular values, with what roundings add "
                                                        "to them, grow past 2^20");
        at += pair ? 2 : 1;
        const bool last = at == n_steps;
        const int eN = exponent_for_largest(std::sqrt(next));
        Product* p = product(last ? Kind::kFinal : Kind::kApply, q, from, last ? kNone : kX,
                             pow2((last ? 0 : eN) - eQ - eX));
        p->out_t = last ? kNone : to;
        // What rounding X left grows with the steps in directions that X hardly has (by 3.44 a step of the usual ones). An
        // apply adds Q's diagonal times it: Q is a, or a a', plus parts along the directions that X has, which meet little
        // of it. The whole Q times it would cost another product. (Five usual steps emulated on 200 x 260, singly after the
        // first pair, without it and with: 32 directions over a floor of 1e-3 8.9e-3 and 2.7e-3, rank 1 1.4e-2 and 3.7e-3, a normal
        // matrix 1.1e-3 both. Measured, it takes 0.19 ms more of 1.64 in an apply of two 8192 x 8192.)
        // It is kept only for steps that together still multiply by more than 4: of the last X's rounding, 2.8e-4 of it, a usual
        // step makes 1e-3.
        p->low_in = kept;
        double ahead = 1.0;
        for (int32_t i = at; i < n_steps; ++i) ahead *= std::max(std::fabs(taken[3 * i]), 1.0);
        kept = p->low_out = !last && ahead > 4.0;
        p->kappa_power = first ? 1 : 0;
        std::swap(from, to);
        eX = eN;
        top = next * (1.0 + kSlack);
    }
    return ZERO_OK;
}

bool make_short_program(const double* coefficients, int32_t n_steps, ShortProgram* out) {
    *out = ShortProgram{};
    if (!steady(coefficients, n_steps, kShortSlack)) return false;
    out->n_steps = n_steps;
    // Eigenvalues of A and of Q, carried through the steps: evenly spaced ones, and as many from 1e-12 up at equal ratios,
    // which cover every interval that small ones grow into.
    constexpr int kCarried = kSamples, kHalf = kCarried / 2, kLanes = 8;
    double x[kCarried], q[kCarried];
    double small = 1.0;
    const double ratio = std::pow(10.0, -12.0 / kHalf);
    for (int i = 0; i < kHalf; ++i, small *= ratio) {
        x[i] = static_cast<double>(i) / kHalf;
        x[kHalf + i] = small;
        q[i] = q[kHalf + i] = 1.0;
    }
    double top = 1.0 + kShortSlack, growth = 1.0;
    int eA = exponent_for_largest(top), eQ = 0;
    out->first = std::ldexp(1.0, eA);
    for (int32_t at = 0; at < n_steps; ++at) {
        const Step step = step_at(coefficients, at);
        const double most_c = step.largest_factor(top), most_t = step.largest_times_x(top), most_a = step.largest_left(top);
        double lanes[kLanes] = {};
        for (int i = 0; i < kCarried; i += kLanes)
            for (int k = 0; k < kLanes; ++k) {
                const double p = step.at(x[i + k]);
                x[i + k] *= p * p;
                q[i + k] *= p;
                lanes[k] = std::max(lanes[k], std::fabs(q[i + k]));
            }
        const double most_q = *std::max_element(lanes, lanes + kLanes);
        // small negative eigenvalues, which roundings make, grow by a^2
        if (at + 1 < n_steps) growth *= std::max(1.0, most_c * most_c);
        if (!(most_c <= 0x1p60) || !(growth <= 65536.0) || !(most_a <= 1024.0) || !(most_q <= 65536.0)) return false;
        const int eC = exponent_for_largest(most_c), eT = exponent_for_largest(most_t), eN = exponent_for_largest(most_a),
                  eP = at == 0 ? eC : exponent_for_largest(most_q);
        ShortStep& s = out->step[at];
        s.a = static_cast<float>(step.a * pow2(eC));
        s.b = static_cast<float>(step.b * pow2(eC - eA));
        s.c = static_cast<float>(step.c * pow2(eC - 2 * eA));
        s.t = pow2(eT - eC - eA);
        s.next = pow2(eN - eT - eC);
        s.q = pow2(eP - eC - eQ);
        eA = eN;
        eQ = eP;
        top = most_a * (1.0 + kShortSlack);
    }
    out->last = pow2(-eQ);
    return true;
}

int32_t short_parts(int32_t side, int64_t n, int64_t count) {
    const int64_t chunks = (n + 63) / 64;
    const double per = side == 64 ? 2.4 : side == 96 ? 1.6 : 1.2, least = side == 64 ? 16 : side == 96 ? 12 : 8;
    const int64_t parts = static_cast<int64_t>(std::max(least, per * std::sqrt(static_cast<double>(chunks))));
    const int64_t room = std::max<int64_t>(1, 2048 / std::max<int64_t>(count, 1));
    return static_cast<int32_t>(std::min({chunks, parts, room, int64_t(256)}));
}

namespace {

constexpr int64_t kTiles[kTileSizes] = {64, 128, 192, 256};

// Microseconds on MI355X of one product: a launch with its descriptors and first loads, each tile's epilogue, and a
// stage of a tile alone on its compute unit or as a share of a full one. Against traces of 487 x 1000, 12 of 768 x 768, 14,336 x
// 4096, two 768 x 2304 and 8192 x 8192, lists of 6 and 12 of two GPTs and 7 of Llama's: square products within 10 %, but for
// lists whose matrices have unlike sides (12 of the 1.3 B GPT: X X^T 299 us for 358, others 114 for 130; Llama's 302 for 340 to
// 360), applies, whose epilogue also keeps and adds what rounding leaves, within 12 %, but for the last one of an update (20 to 50 %
// more, its 10 bytes an element).
struct TileCost {
    double launch, tile, alone, share;
};
constexpr TileCost kSquareCosts[kTileSizes] = {
    {5.0, 0.6, 0.30, 0.23}, {6.0, 2.0, 0.62, 0.52}, {3.0, 6.0, 0.96, 1.02}, {3.0, 9.0, 1.18, 1.45}};
constexpr TileCost kApplyCosts[kTileSizes] = {
    {5.0, 2.0, 0.30, 0.23}, {6.0, 4.5, 0.62, 0.52}, {}, {3.0, 34.0, 1.18, 1.45}};        // (no applies with 192)

double product_time(const TileCost& c, double tiles, double stages) {
    if (tiles == 0.0) return 0.0;
    const double load = std::ceil(tiles / kUnits);       // tiles of one compute unit
    return c.launch + c.tile * load + stages / tiles * (load > 1.0 ? std::max(c.alone, c.share * load) : c.alone);
}

// Of a square product's tiles kTiles[k].
double square_time(int k, double tiles, double stages) {
    if (kTiles[k] == 256 && tiles < 1e9) {
        const double whole = whole_tiles(static_cast<uint32_t>(tiles));
        if (whole < tiles) {
            const double each = stages / tiles;          // a quarter of a tile is one of 128, alone on its unit
            return product_time(kSquareCosts[k], whole, each * whole) + kSquareCosts[1].tile + each * kSquareCosts[1].alone;
        }
    }
    return product_time(kSquareCosts[k], tiles, stages);
}

int64_t padded(int64_t side, int64_t tile) { return std::max(pad(side, 64), tile); }

}  // namespace

void TileChoice::add(int64_t count, int64_t rows, int64_t cols) {
    const int64_t least = std::min(rows, cols), most = std::max(rows, cols);
    for (int k = 0; k < kTileSizes; ++k) {
        for (int j = 0; j < kTileSizes; ++j) {
            const int64_t ts = kTiles[k], tr = kTiles[j], M = padded(least, std::max(ts, tr)),
                          N = padded(most, std::max(ts, tr)), across = (M + ts - 1) / ts;
            const double c = static_cast<double>(count), square = c * (across * (across + 1) / 2),
                         rect = c * ((M + tr - 1) / tr) * ((N + tr - 1) / tr);
            Total& x = total_[k][j];
            x.square += square;
            x.rect += rect;
            x.gram += square * (N / 64);
            x.squares += square * (M / 64);
            x.apply += rect * (M / 64);
        }
    }
}

void TileChoice::best(int64_t* square, int64_t* rect, Times* times) const {
    double least = 0.0;
    *square = *rect = 0;
    for (int k = 0; k < kTileSizes; ++k) {
        for (int j = 0; j < kTileSizes; ++j) {
            if (kTiles[j] == 192) continue;
            const Total& x = total_[k][j];
            const Times t{square_time(k, x.square, x.gram), square_time(k, x.square, x.squares),
                          product_time(kApplyCosts[j], x.rect, x.apply)};
            const double time = program_time(t, 5, true);
            if (*square == 0 || time < least) {
                *square = kTiles[k];
                *rect = kTiles[j];
                *times = t;
                least = time;
            }
        }
    }
}

void shape(Desc* d, int64_t rows, int64_t cols, int64_t tile) {
    const int64_t numel = rows * cols;
    d->rows = static_cast<int32_t>(rows);
    d->cols = static_cast<int32_t>(cols);
    d->M = static_cast<int32_t>(padded(std::min(rows, cols), tile));
    d->N = static_cast<int32_t>(padded(std::max(rows, cols), tile));
    d->chunk = std::max(kChunk, pad((numel + kMaxChunks - 1) / kMaxChunks, kChunk));
    d->chunks = static_cast<int32_t>((numel + d->chunk - 1) / d->chunk);
}

int64_t grid_count(const Desc& d, int grid, int64_t square_tile, int64_t rect_tile) {
    const int64_t across = (d.M + square_tile - 1) / square_tile;
    switch (grid) {
        case kByChunk: return d.chunks;
        case kByPack: return (d.M / kPack) * (d.N / kPack);
        case kByTile: return ((d.M + rect_tile - 1) / rect_tile) * ((d.N + rect_tile - 1) / rect_tile);
        case kByPart: return d.parts;
        default: return across * (across + 1) / 2;
    }
}

int64_t area_bytes(const Desc& d) {
    const int64_t m = d.M, n = d.N, ldm = stride(d.M), ldn = stride(d.N);
    return pad(2 * (m * ldn + 2 * n * ldm + 3 * m * ldm + std::max(m * ldn, n * ldm)), 256);
}

int64_t head_bytes(int64_t partials, int64_t matrices) { return pad(8 * partials + 4 * matrices, 256); }

}  // namespace muon
}  // namespace zero
