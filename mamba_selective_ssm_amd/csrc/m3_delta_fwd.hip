// Gated delta rule, prefill: chunk matrices, then the walk over the chunks.
#include "m3_delta_chunk.hpp"
#include "m3_delta_wide.hpp"

namespace m3 {

namespace {

template <typename IO, int N>
hipError_t fwd_n(const DeltaParams& p, hipStream_t stream)
{
    const hipError_t e = launch_delta_chunks<IO, N, false>(p, stream);
    if (e != hipSuccess) return e;
    if constexpr (sizeof(IO) == 2) {
        if ((int64_t)p.rows * p.H * (p.P / 16) > 256) {
            if constexpr (N < 128)
                if (p.P % 64 == 0) return launch_delta_wide<N, 4>(p, stream);
            return launch_delta_wide<N, 2>(p, stream);
        }
    }
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
