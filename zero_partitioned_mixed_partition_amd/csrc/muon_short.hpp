// The launches for matrices with a short side of at most 128 (muon_short.hip).
#pragma once

#include "muon_device.hpp"

namespace zero {
namespace muon {

// Runs the program on matrices whose short sides are all at most m.side. source: 0 bf16, 1 fp32, 2 momentum
// and gradient with the weight update.
zero_status launch_short(int source, const dev::Matrices& m, const dev::MomentumScalars& s,
                         const dev::Update& u, const ShortProgram& program, double eps, hipStream_t stream, const char* who);

}  // namespace muon
}  // namespace zero
