// Gated delta rule, one token per row on a resident float32 state.
//
//   p = a S^T k,  u = beta (v - p),  S <- a S + k u^T,
//   o = scale S^T q = scale (a S_old^T q + u (k.q))
//
// The state is read and written once (8 N P bytes a head) against 7 N P
// operations: bound by memory.  The second form of o lets one pass over the
// old state make both sums, so a wavefront holds its part in registers,
// updates it there and stores it: no second read.  One wavefront takes 32
// columns (128 bytes of each state row) of one head; lane (rg, cq) holds rows
// rg N/8 .. +N/8-1 of columns 4 cq .. +3, so its k and q values are contiguous
// too.  All its loads are in flight at once (N/8 of 16 bytes a lane), and the
// only exchange is the sum over the eight row groups.
// 256 rows x 32 heads, N = 128, P = 64, 537 MB of state read and written: calls in
// turn on four states 110 us, 4.9 TB/s (a copy of 4 GiB runs at 4.7); one after the
// other on one, part of which then lies in the caches, 84.  Loads that bypass the
// caches: 108 and 85, one or two wavefronts to a workgroup instead of four: 113 and
// 88, 113 and 85.
// A row in a slot first looks for its slot in all earlier rows' entries, beside its
// loads: 2 us of 51 at 256 rows, 15 of 229 at 4096, 260 of 1109 at 16384 (8 heads, N
// = P = 64).
#include "m3_delta.hpp"

namespace m3 {

namespace {

constexpr int kStepWaves = 4;

// As delta_record, for one wavefront.
__device__ __forceinline__ int64_t step_record(const DeltaParams& p, int b, int lane)
{
    if (p.slots == nullptr) return b;
    const int s = p.slots[b];
    bool seen = false;
    for (int i = lane; i < b; i += 64) seen |= p.slots[i] == s;
    if (s < 0 || s >= p.nslots) return -1;
    return __any(seen) ? -2 : s;
}

__device__ __forceinline__ void load4(float (&d)[4], const bf16* p)
{
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = (float)v[e];
}
__device__ __forceinline__ void load4(float (&d)[4], const float* p)
{
    const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = v[e];
}

__device__ __forceinline__ float groups_sum(float v)
{
    v += __shfl_xor(v, 8);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

template <typename IO, int N>
__global__ __launch_bounds__(64 * kStepWaves) void delta_step_kernel(const DeltaParams p)
{
    constexpr int RN = N / 8;
    const int lane = threadIdx.x & 63, rg = lane >> 3, cq = lane & 7;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nsl = p.P / 32;
    const int64_t unit = (int64_t)blockIdx.x * kStepWaves + wv;
    if (unit >= (int64_t)p.rows * p.H * nsl) return;   // whole wavefront
    const int64_t bh = unit / nsl;
    const int p0 = (int)(unit % nsl) * 32 + 4 * cq;
    int64_t b, h;
    split_bh(bh, p.H, b, h);
    const int64_t rec = step_record(p, (int)b, lane);
    const int64_t qk = (b * p.G + h / (p.H / p.G)) * N + rg * RN;
    float* hs = p.h_out + ((rec * p.H + h) * N + rg * RN) * p.P + p0;

    f32x4 S[RN];
#pragma unroll
    for (int i = 0; i < RN; ++i) {
        S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (rec >= 0) S[i] = *reinterpret_cast<const f32x4*>(hs + (int64_t)i * p.P);
    }
    float k[RN], q[RN];
#pragma unroll
    for (int i = 0; i < RN; i += 4) {
        float t[4];
        load4(t, reinterpret_cast<const IO*>(p.k) + qk + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) k[i + e] = t[e];
        load4(t, reinterpret_cast<const IO*>(p.q) + qk + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) q[i + e] = t[e];
    }
    float v[4];
    load4(v, reinterpret_cast<const IO*>(p.v) + bh * p.P + p0);
    const float a = expf(p.g[bh]), beta = p.beta[bh];

    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < RN; ++i) {
        kk += k[i] * k[i];
        qq += q[i] * q[i];
        kq += k[i] * q[i];
    }
    kq = groups_sum(kq);
    float rk = 1.f, rq = p.scale;
    if (p.l2norm) {
        rk = 1.f / sqrtf(groups_sum(kk) + p.eps);
        rq *= 1.f / sqrtf(groups_sum(qq) + p.eps);
    }
    f32x4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
#pragma unroll
    for (int i = 0; i < RN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] += S[i][e] * k[i];
            sq[e] += S[i][e] * q[i];
        }
    f32x4 u, o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float pk = a * groups_sum(sk[e]) * rk;
        u[e] = beta * (v[e] - pk);
        o[e] = rq * (a * groups_sum(sq[e]) + u[e] * (kq * rk));
        u[e] *= rk;
    }
    if (rec == -2) {   // the record belongs to an earlier row
        const float nan = __builtin_nanf("");
        o = f32x4{nan, nan, nan, nan};
    }
    if (rec >= 0)
#pragma unroll
        for (int i = 0; i < RN; ++i) {
            f32x4 n;
#pragma unroll
            for (int e = 0; e < 4; ++e) n[e] = a * S[i][e] + k[i] * u[e];
            *reinterpret_cast<f32x4*>(hs + (int64_t)i * p.P) = n;
        }
    if (rg == 0) gstore4(reinterpret_cast<IO*>(p.o) + bh * p.P + p0, o);
}

template <typename IO, int N>
hipError_t step_n(const DeltaParams& p, hipStream_t stream)
{
    const int64_t units = (int64_t)p.rows * p.H * (p.P / 32);
    hipLaunchKernelGGL((delta_step_kernel<IO, N>), dim3((unsigned)((units + kStepWaves - 1) / kStepWaves)),
                       dim3(64 * kStepWaves), 0, stream, p);
    return hipGetLastError();
}

template <typename IO>
hipError_t step_io(const DeltaParams& p, hipStream_t stream)
{
    switch (p.N) {
    case 32: return step_n<IO, 32>(p, stream);
    case 64: return step_n<IO, 64>(p, stream);
    default: return step_n<IO, 128>(p, stream);
    }
}

}  // namespace

hipError_t launch_delta_step(const DeltaParams& p, int io_dtype, hipStream_t stream)
{
    return io_dtype == 0 ? step_io<float>(p, stream) : step_io<bf16>(p, stream);
}

}  // namespace m3
