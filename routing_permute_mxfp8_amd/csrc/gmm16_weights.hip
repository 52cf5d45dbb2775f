#include "gmm16_tile.h"

namespace moe {
hipError_t launch_gmm16_weights(const Gmm16Params& p, hipStream_t stream) { return launch_tile16_form<kWeights>(p, stream); }
}  // namespace moe
