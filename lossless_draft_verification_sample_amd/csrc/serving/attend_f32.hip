// The attention kernel for float32 queries.

#include "attend_kernel.hpp"

namespace sv {

int launch_attend_f32(const AttendArgs& a, hipStream_t st) { return launch_attend_typed<true>(a, st); }

}  // namespace sv
