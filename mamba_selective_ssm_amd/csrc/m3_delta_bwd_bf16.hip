// Gated delta rule, gradient, bfloat16.
#include "m3_delta_back.hpp"

namespace m3 {

hipError_t launch_delta_bwd_bf16(const DeltaBwdParams& p, hipStream_t stream) { return launch_delta_bwd_io<bf16>(p, stream); }

}  // namespace m3
