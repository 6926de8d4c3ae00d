#include "m3_delta_chunk.hpp"
namespace m3 { hipError_t launch_delta_bwd(const DeltaBwdParams&, int, hipStream_t) { return hipErrorNotSupported; } }
