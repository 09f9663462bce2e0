// Prints the products and the short-side program that the Muon planner makes for coefficients (muon_plan.hpp).
// Arguments: "tiled" <pairs 0/1> <low 0/1> or "short", then a, b, c of each step. Output: the status, and per product its kind
// and factors; or whether there is a short-side program, and per step its factors.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "muon_plan.hpp"

int main(int argc, char** argv) {
    using namespace zero::muon;
    const bool tiled = argc > 1 && std::strcmp(argv[1], "tiled") == 0;
    const int from = tiled ? 4 : 2;
    std::vector<double> steps;
    for (int i = from; i < argc; ++i) steps.push_back(std::strtod(argv[i], nullptr));
    const int32_t n = static_cast<int32_t>(steps.size() / 3);
    if (tiled) {
        std::vector<Product> program;
        const zero_status st = make_program(steps.data(), n, std::atoi(argv[2]) != 0, std::atoi(argv[3]) != 0, &program, "steps");
        std::printf("%d %s\n", static_cast<int>(st), zero_last_error());
        if (st != ZERO_OK) return 0;
        for (const Product& p : program)
            std::printf("%d %d %d %d %d %d %d %d %d %.9g %.9g %.9g\n", static_cast<int>(p.kind), p.lhs, p.rhs, p.add, p.out,
                        p.kappa_power, p.low_in, p.low_out, p.full, p.alpha, p.beta, p.diag);
        return 0;
    }
    ShortProgram program;
    const bool ok = make_short_program(steps.data(), n, &program);
    std::printf("%d\n", ok ? 1 : 0);
    if (!ok) return 0;
    std::printf("%.17g %.9g\n", program.first, program.last);
    for (int32_t i = 0; i < program.n_steps; ++i) {
        const ShortStep& s = program.step[i];
        std::printf("%.9g %.9g %.9g %.9g %.9g %.9g\n", s.a, s.b, s.c, s.t, s.next, s.q);
    }
    return 0;
}
