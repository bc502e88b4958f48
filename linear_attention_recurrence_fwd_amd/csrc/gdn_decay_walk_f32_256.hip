// Walks of the decay operator over up to 256 channels, f32 tensors.
#include "gdn_decay_walk.h"

namespace gdn {
hipError_t decay_walk_f32_256(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_kd<float, 256>(a, st); }
hipError_t decay_sum_f32_256(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_sum_kd<float, 256>(a, st); }
}  // namespace gdn
