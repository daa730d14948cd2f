// kda_linear_rev_f32.hip -- the backward walks of kda_linear_walk.hpp for f32 elements (one of four files
// that compile side by side).
#include <type_traits>

#include "kda_linear_walk.hpp"

namespace kda {
hipError_t launch_linear_rev_f32(const LinearArgs& a, hipStream_t st) { return launch_walk_t<float, true>(a, st); }
}  // namespace kda
