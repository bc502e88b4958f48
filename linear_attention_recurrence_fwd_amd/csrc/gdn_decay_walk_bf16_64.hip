// Walks of the decay operator over up to 64 channels, bf16 tensors.
#include "gdn_decay_walk.h"

namespace gdn {
hipError_t decay_walk_bf16_64(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_kd<bf16, 64>(a, st); }
hipError_t decay_sum_bf16_64(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_sum_kd<bf16, 64>(a, st); }
}  // namespace gdn
