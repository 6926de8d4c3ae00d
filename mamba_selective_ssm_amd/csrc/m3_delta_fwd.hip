// Gated delta rule, prefill: chunk matrices, then the walk over the chunks.
#include "m3_delta_chunk.hpp"
#include "m3_delta_wide.hpp"

namespace m3 {

namespace {

// A part of every row's chunks is walked beside the next part's chunk matrices:
// workgroups [0, walks) have the walk, each wavefront of the others a chunk and
// head.  The walk alone leaves the CUs idle that it has no slices for.
template <typename IO, int N>
__global__ __launch_bounds__(64 * 8) void delta_both_kernel(const DeltaParams p, const DeltaParams next, const unsigned walks)
{
    extern __shared__ __attribute__((aligned(16))) char wlds[];
    if (blockIdx.x < walks) {
        delta_walk<IO, N, false>(p, nullptr, nullptr, blockIdx.x, wlds);
        return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)(blockIdx.x - walks) * 8 + wave;
    if (unit < (int64_t)next.rows * next.nc * next.H) delta_chunk<IO, N, false>(next, unit, wlds + wave * kChunkLds);
}

template <typename IO, int N>
hipError_t launch_delta_parts(const DeltaParams& p, hipStream_t stream)
{
    using Cf = WalkCfg<IO, N, false>;
    static_assert(Cf::waves == 8, "a wavefront to each of delta_both_kernel's chunks");
    constexpr size_t lds = Cf::total > 8 * kChunkLds ? Cf::total : 8 * kChunkLds;
    static_assert(lds <= 160 * 1024, "a workgroup's LDS");
    auto* const kern = &delta_both_kernel<IO, N>;
    static std::atomic<uint64_t> done{0};
    hipError_t e = delta_allow_lds(kern, lds, done);
    if (e != hipSuccess) return e;
    const int64_t each = delta_part((int64_t)p.rows * p.H, sizeof(IO) == 4 ? 0 : 1);
    auto part = [&](int64_t from) {
        DeltaParams q = p;
        q.from = from;
        q.count = each;
        q.nc = (int)(p.nc - from < each ? p.nc - from : each);
        if (from == 0) q.carry_in = nullptr;
        if (from + each >= p.nc) q.carry_out = nullptr;
        return q;
    };
    if ((e = launch_delta_chunks<IO, N, false>(part(0), stream)) != hipSuccess) return e;
    const unsigned walks = (unsigned)(((int64_t)p.rows * p.H + 7) / 8 * 8 * (p.P / 16));
    for (int64_t c = 0; c < p.nc; c += each) {
        const DeltaParams now = part(c);
        DeltaParams next = now;
        next.nc = 0;
        if (c + each < p.nc) next = part(c + each);
        const unsigned chunks = (unsigned)(((int64_t)p.rows * next.nc * p.H + 7) / 8);
        hipLaunchKernelGGL(kern, dim3(walks + chunks), dim3(64 * 8), lds, stream, now, next, walks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

// Which walk.  A slice is 16 columns of one row and head.  Up to one slice per
// CU its chain of products is the call's time, and four wavefronts on one slice
// (delta_walk) take less than one wavefront's registers (delta_wide): 72 against
// 94 us a call at 256 slices, 2048 tokens, N = 64.  With more, a CU's LDS reads
// are, and delta_wide has a quarter of them (whole calls over 2048 tokens, us, P =
// 64, delta_walk / delta_wide): N = 64: 288 slices 118 / 107, 384: 123 / 111,
// 512: 136 / 123, 768: 261 / 189, 1024: 334 / 228; N = 32, 512: 116 / 98; N =
// 128, 288: 139 / 123, 512: 185 / 155, 1024: 369 / 269.  Where P allows, 64
// columns go to a workgroup above 512 slices: with 32 of them such calls are two
// rounds over the chip or more (N = 64: 544 slices 170 for 142, 768: 231 for
// 189, 1024: 264 for 228; N = 128, 1024: 314 for 269).  Up to there half of the
// CUs would be idle with 64 (N = 64, 512 slices: 137 for 123; N = 128: 173 for 155).
template <typename IO, int N>
hipError_t fwd_n(const DeltaParams& p, hipStream_t stream)
{
    if (p.carry_out != nullptr) return launch_delta_parts<IO, N>(p, stream);
    const hipError_t e = launch_delta_chunks<IO, N, false>(p, stream);
    if (e != hipSuccess) return e;
    if constexpr (sizeof(IO) == 2) {
        const int64_t slices = (int64_t)p.rows * p.H * (p.P / 16);
        if (slices > 256) {
            if (p.P % 64 == 0 && slices > 512) return launch_delta_wide<N, 4>(p, stream);
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
