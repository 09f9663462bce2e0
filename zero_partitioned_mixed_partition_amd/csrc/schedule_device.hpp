// A step schedule's device-resident state, shared by the translation units
// whose kernels read it (the 32-bit and the 8-bit AdamW).
#pragma once

#include <cstdint>

#include "schedule.hpp"

namespace zero {
namespace adam {

// A step schedule's device state: the scalars of the next step to apply and
// the number of updates applied so far. The scheduled AdamW reads `next`; the
// advance kernel, once per step, moves both on.
struct alignas(64) AdamState {
    StepScalars next;
    int64_t applied;
    int64_t unused[3];
};
static_assert(sizeof(AdamState) == 64, "one 64-byte state");

// ZERO_EINVAL unless the schedule lives on the current device.
zero_status check_schedule_device(const zero_adamw_schedule* schedule, const char* who);

}  // namespace adam
}  // namespace zero

struct zero_adamw_schedule {
    int device = -1;
    void* mem = nullptr;               // the state, then the table
    zero::adam::AdamState* state = nullptr;
    const zero::adam::StepScalars* table = nullptr;
    int64_t length = 0;
};
