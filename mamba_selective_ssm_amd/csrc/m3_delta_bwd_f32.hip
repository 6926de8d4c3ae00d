// Gated delta rule, gradient, float32.
#include "m3_delta_back.hpp"

namespace m3 {

hipError_t launch_delta_bwd_f32(const DeltaBwdParams& p, hipStream_t stream) { return launch_delta_bwd_io<float>(p, stream); }

}  // namespace m3
