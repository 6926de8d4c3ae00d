// Gated delta rule, prefill: chunk matrices, then the walk over the chunks.
#include "m3_delta_chunk.hpp"
#include "m3_delta_walk.hpp"

namespace m3 {

namespace {

template <typename IO, int N>
hipError_t fwd_n(const DeltaParams& p, hipStream_t stream)
{
    const hipError_t e = launch_delta_chunks<IO, N, false>(p, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    return launch_delta_walk<IO, N>(p, stream);
}

template <typename IO>
hipError_t fwd_io(const DeltaParams& p, hipStream_t stream)
{
    switch (p.N) {
    case 32: return fwd_n<IO, 32>(p, stream);
    case 64: return fwd_n<IO, 64>(p, stream);
    default: return fwd_n<IO, 128>(p, stream);
    }
}

}  // namespace

hipError_t launch_delta_fwd(const DeltaParams& p, int io_dtype, hipStream_t stream)
{
    return io_dtype == 0 ? fwd_io<float>(p, stream) : fwd_io<bf16>(p, stream);
}

}  // namespace m3
