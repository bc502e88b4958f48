// dq and dk of the decay operator, bf16, value heads of up to 256 channels.
#include "gdn_decay_keys.h"

namespace gdn {
hipError_t decay_keys_256(const DecayKeysArgs& a, hipStream_t st) { return decay::launch_keys<256>(a, st); }
}  // namespace gdn
