// Walks of the decay operator over up to 192 channels, bf16 tensors.
#include "gdn_decay_walk.h"

namespace gdn {
hipError_t decay_walk_bf16_192(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_kd<bf16, 192>(a, st); }
hipError_t decay_sum_bf16_192(const DecayWalkArgs& a, hipStream_t st) { return decay::launch_sum_kd<bf16, 192>(a, st); }
}  // namespace gdn
