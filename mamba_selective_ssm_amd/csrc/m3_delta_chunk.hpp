// Gated delta rule: the kernel that makes what a chunk's products need and no
// state enters: T, A and per-token factors.
#pragma once

#include "m3_delta.hpp"

namespace m3 {

// acc += A B for 16 x 16 float32 tiles in LDS (row-major, leading dimension
// LD): lane (l, g) supplies A[l][k], B[k][l] of k = 4 kk + g.
template <int LD>
__device__ __forceinline__ void tile_mm(const float* A, const float* B, int l, int g, f32x4& acc)
{
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(A[l * LD + 4 * kk + g], B[(4 * kk + g) * LD + l], acc, 0, 0, 0);
}
template <int LD>
__device__ __forceinline__ void tile_put(float* C, int l, int g, const f32x4& v)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) C[(4 * g + r) * LD + l] = v[r];
}

// Inclusive prefix sum across a wavefront in float64, by the lane moves of
// wave_inclusive_sum on both halves.
template <int CTRL, int ROW_MASK> __device__ __forceinline__ double dpp_moved_d(double x)
{
    const long long b = __builtin_bit_cast(long long, x);
    const unsigned lo = (unsigned)dpp_moved_i<CTRL, ROW_MASK>((int)(b & 0xffffffffll));
    const unsigned hi = (unsigned)dpp_moved_i<CTRL, ROW_MASK>((int)(b >> 32));
    return __builtin_bit_cast(double, (long long)(((unsigned long long)hi << 32) | lo));
}
__device__ __forceinline__ double wave_inclusive_sum_d(double v)
{
    v += dpp_moved_d<0x111, 0xf>(v);
    v += dpp_moved_d<0x112, 0xf>(v);
    v += dpp_moved_d<0x114, 0xf>(v);
    v += dpp_moved_d<0x118, 0xf>(v);
    v += dpp_moved_d<0x142, 0xa>(v);
    v += dpp_moved_d<0x143, 0xc>(v);
    return v;
}

// Sum over each 16 lanes in float64, by the lane moves of lane_group_sum.
__device__ __forceinline__ double lane_group_sum_d(double v)
{
    v += dpp_moved_d<0xB1, 0xf>(v);
    v += dpp_moved_d<0x4E, 0xf>(v);
    v += dpp_moved_d<0x141, 0xf>(v);
    v += dpp_moved_d<0x140, 0xf>(v);
    return v;
}

// The operand blocks of a lower triangular matrix in LDS: block (w, kb) has
// rows tile_row(w, l), columns 32 kb + 8 g ..+7; zero above the diagonal.  f(block,
// its two halves of 4 columns).
template <int LD, typename F> __device__ __forceinline__ void each_lower(const float* M, int l, int g, const F& f)
{
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int kb = 0; kb <= w / 2; ++kb) {
            const int row = tile_row(w, l), c0 = 32 * kb + 8 * g;
            f32x4 a = *reinterpret_cast<const f32x4*>(M + row * LD + c0);
            f32x4 b = *reinterpret_cast<const f32x4*>(M + row * LD + c0 + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = c0 + e <= row ? a[e] : 0.f;
                b[e] = c0 + 4 + e <= row ? b[e] : 0.f;
            }
            f(low_block(w, kb), a, b);
        }
}

// What one chunk of one head needs besides its rows:
//   T = (I + M)^-1, A = scale D o Q K^T (rows divided by their norms where the
//   call asks for it), and per token  beta | beta e^G / |k| | e^(G_last - G) /
//   |k| | scale e^G / |q| | e^G_last.
// BWD: without A and the last but one, with 1 / |k| | G's two parts instead.
// One wavefront per chunk and head, on its own: no barriers, and the steps
// that wait on each other (the sums over the chunk, the inverse) run beside
// those of the other wavefronts on the SIMD.  K and Q rows are the operands as
// they lie in memory (lane: one row, 8 columns), so the two 64 x 64 products
// take no LDS.  M is inverted by blocks, in place: substitution inside the
// four 16 x 16 diagonal blocks (lane (l, g): column l of block g, in
// registers), then pairs of blocks joined, [[A,0],[C,B]]^-1 = [[A^-1,0],
// [-B^-1 C A^-1, B^-1]], with float32 matrix instructions; C A^-1 waits in the
// unused block above the diagonal.  Substitution and not the product
// (I-M)(I+M^2)(I+M^4).., whose terms cancel where keys repeat.  G is summed in
// 64 bits and kept as two float32 in units of log 2: the difference of two
// sums keeps float32's relative precision after a token whose decay is near
// zero.  Rows past the end read the last row again; their beta is 0 and their
// g is 0, which makes their rows of T the identity's.
// Bound by memory: at N = 64 in bf16 16 KB of rows come in and 31 KB of T (three
// planes), A (float32) and factors go out per chunk and head, 63 KB at N = 128.  20 us for 2048
// chunks and heads at N = 64 (4.7 TB/s), 424 us for 32768 at N = 128 (4.9
// TB/s), 16 us for the gradient's 28 KB each (2048; 3.6 TB/s).  A workgroup of
// four wavefronts with shared rows and barriers took 40 and 750 us.  Without A,
// which the walk would then make, 15.6 and 246 us; but the walk lost more (56
// for its 39 of then and 1980 for 1660 us).
constexpr int kChunkLds = (64 * 68 + 5 * 64) * 4;   // bytes
template <typename IO, int N, bool BWD>
__device__ __forceinline__ void delta_chunk(const DeltaParams& p, int64_t bid, char* lds)
{
    constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide;
    constexpr int KB = N / 32, LD = 68;
    float* sM = reinterpret_cast<float*>(lds);
    float *sGh = sM + 64 * LD, *sGl = sGh + 64, *sBk = sGl + 64, *sRk = sBk + 64, *sRq = sRk + 64;

    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int h = (int)(bid % p.H);
    const int bc = (int)(bid / p.H);
    int b, c;
    delta_place(p, bc, b, c);
    if (bid < p.rows && p.from == 0 && p.order != nullptr) delta_rank(p, (int)bid, lane);   // (as many as rows run, at least)
    const DeltaRow row = delta_row(p, b);
    if ((int64_t)c * kDC >= row.len) return;
    const int64_t t0 = row.start + (int64_t)c * kDC;
    const int nv = row.len - (int64_t)c * kDC < kDC ? (int)(row.len - (int64_t)c * kDC) : kDC;
    const int64_t ci = (row.slot0 + c) * p.H + h;
    const int hg = h / (p.H / p.G);
    const IO* kp = reinterpret_cast<const IO*>(p.k) + (t0 * p.G + hg) * N;
    const IO* qp = reinterpret_cast<const IO*>(p.q) + (t0 * p.G + hg) * N;
    const int rs = p.G * N;   // row stride of q and k

    const int tok = lane < nv ? lane : nv - 1;
    float gv = p.g[(t0 + tok) * p.H + h];
    float bv = p.beta[(t0 + tok) * p.H + h];
    RawRow8<IO> kr[4][KB], qr[4][KB];
    int off[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        const int i = 16 * rt + l < nv ? 16 * rt + l : nv - 1;
        off[rt] = i * rs + 8 * g;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) kr[rt][kb].load(kp + off[rt] + 32 * kb, true);
    }
    // the larger rows would not fit beside K's: they are read tile by tile
    constexpr bool ALLQ = KP == 1 && N < 128;
#pragma unroll
    for (int rt = 0; rt < (BWD ? 0 : ALLQ ? 4 : 1); ++rt)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) qr[rt][kb].load(qp + off[rt] + 32 * kb, true);

    const bool real = lane < nv;
    gv = real ? (gv < -1024.f ? -1024.f : gv) : 0.f;   // exp is zero there; keeps -inf out of differences
    bv = real ? bv : 0.f;
    const double G = wave_inclusive_sum_d((double)gv * 1.4426950408889634);
    const double Gl = __shfl(G, 63);
    const float gh = (float)G;
    const float eG = __builtin_amdgcn_exp2f(gh), dG = __builtin_amdgcn_exp2f((float)(Gl - G));
    sGh[lane] = gh;
    sGl[lane] = (float)(G - (double)gh);

    // K K^T, tiles on and below the diagonal
    f32x4 kk[4][4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int ct = 0; ct <= rt; ++ct) kk[rt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            bf16x8 j[KP];
            kr[ct][kb].planes(j);
#pragma unroll
            for (int rt = ct; rt < 4; ++rt) {
                bf16x8 a[KP];
                kr[rt][kb].planes(a);
                mma_planes<KP, KP, WP>(a, j, kk[rt][ct]);
            }
        }
    float rk = 1.f;
    if (p.l2norm) {   // |k|^2 is the diagonal
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (l == 4 * g + r) sRk[16 * rt + l] = kk[rt][rt][r];
        wave_order();
        rk = __builtin_amdgcn_rsqf(sRk[lane] + p.eps);
        wave_order();
    }
    sRk[lane] = rk;
    sBk[lane] = bv * rk;
    wave_order();

    // A = scale D o Q K^T, one row tile at a time
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};
    float cgh[4], cgl[4], crk[4];
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        cgh[ct] = sGh[16 * ct + l];
        cgl[ct] = sGl[16 * ct + l];
        crk[ct] = sRk[16 * ct + l];
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        f32x4 qk[4] = {fz, fz, fz, fz}, rq4 = fz;
        if constexpr (!BWD) {
            float q2 = 0.f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8 a[KP];
                qr[ALLQ ? rt : 0][kb].planes(a);
                if (p.l2norm)
#pragma unroll
                    for (int e = 0; e < 8; ++e) q2 += qr[ALLQ ? rt : 0][kb].get(e) * qr[ALLQ ? rt : 0][kb].get(e);
#pragma unroll
                for (int ct = 0; ct <= rt; ++ct) {
                    bf16x8 j[KP];
                    kr[ct][kb].planes(j);
                    mma_planes<KP, KP, WP>(a, j, qk[ct]);
                }
                if (!ALLQ && rt < 3) qr[0][kb].load(qp + off[rt < 3 ? rt + 1 : 3] + 32 * kb, true);
            }
            if (p.l2norm) {
                q2 += __shfl_xor(q2, 16);
                q2 += __shfl_xor(q2, 32);
                q2 = __builtin_amdgcn_rsqf(q2 + p.eps);
            } else {
                q2 = 1.f;
            }
            if (g == 0) sRq[16 * rt + l] = q2;
            wave_order();
            rq4 = *reinterpret_cast<const f32x4*>(&sRq[16 * rt + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) rq4[r] *= p.scale;
        }
        const f32x4 gh4 = *reinterpret_cast<const f32x4*>(&sGh[16 * rt + 4 * g]);
        const f32x4 gl4 = *reinterpret_cast<const f32x4*>(&sGl[16 * rt + 4 * g]);
        const f32x4 bk4 = *reinterpret_cast<const f32x4*>(&sBk[16 * rt + 4 * g]);
#pragma unroll
        for (int ct = 0; ct <= rt; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool diag = ct == rt;
                const int i = 4 * g + r;   // row in the tile
                float D = __builtin_amdgcn_exp2f((gh4[r] - cgh[ct]) + (gl4[r] - cgl[ct])) * crk[ct];
                if (diag && l > i) D = 0.f;
                if constexpr (!BWD) sM[(16 * rt + i) * LD + 16 * ct + l] = rq4[r] * D * qk[ct][r];
                // D's last use is M: kk becomes M here
                kk[rt][ct][r] = (diag && l >= i) ? 0.f : bk4[r] * D * kk[rt][ct][r];
            }
    }
    {
        float* sc = p.sc + ci * (kDScal * 64) + lane;
        sc[0] = bv;
        sc[64] = bv * eG * rk;
        sc[128] = dG * rk;
        sc[256] = __builtin_amdgcn_exp2f((float)Gl);   // e^G_last, for every lane
        if constexpr (BWD) {
            sc[320] = rk;
            sc[384] = gh;
            sc[448] = sGl[lane];
        } else {
            wave_order();
            sc[192] = p.scale * eG * sRq[lane];
            float* dst = p.af + ci * (int64_t)kTriValues + 4 * lane;
            each_lower<LD>(sM, l, g, [&](int i, const f32x4& a, const f32x4& b) {
                *reinterpret_cast<f32x4*>(dst + 512 * i) = a;
                *reinterpret_cast<f32x4*>(dst + 512 * i + 256) = b;
            });
        }
    }

    // M takes A's place
    wave_order();
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int ct = 0; ct <= rt; ++ct) tile_put<LD>(&sM[16 * rt * LD + 16 * ct], l, g, kk[rt][ct]);
    wave_order();
    // the diagonal blocks: column l of block g
    {
        const float* m0 = &sM[16 * g * LD + 16 * g];
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == l ? 1.f : 0.f;
#pragma unroll
            for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
                const f32x4 m = *reinterpret_cast<const f32x4*>(m0 + i * LD + 4 * j4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * j4 + e < i) s -= m[e] * x[4 * j4 + e];
            }
            x[i] = s;
        }
        wave_order();
#pragma unroll
        for (int i = 0; i < 16; ++i) sM[(16 * g + i) * LD + 16 * g + l] = x[i];
    }
    wave_order();
    // blocks (1,0) and (3,2)
    {
        f32x4 x[2] = {fz, fz};
#pragma unroll
        for (int w = 0; w < 2; ++w) tile_mm<LD>(&sM[(32 * w + 16) * LD + 32 * w], &sM[32 * w * LD + 32 * w], l, g, x[w]);
#pragma unroll
        for (int w = 0; w < 2; ++w) tile_put<LD>(&sM[32 * w * LD + 32 * w + 16], l, g, x[w]);
        wave_order();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[w] = fz;
            tile_mm<LD>(&sM[(32 * w + 16) * LD + 32 * w + 16], &sM[32 * w * LD + 32 * w + 16], l, g, x[w]);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) tile_put<LD>(&sM[(32 * w + 16) * LD + 32 * w], l, g, -x[w]);
    }
    wave_order();
    // the 32 x 32 block below: X = C A^-1, then -B^-1 X
    {
        f32x4 x[2][2] = {{fz, fz}, {fz, fz}};
#pragma unroll
        for (int ta = 0; ta < 2; ++ta)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
#pragma unroll
                for (int k = tb; k < 2; ++k)
                    tile_mm<LD>(&sM[(32 + 16 * ta) * LD + 16 * k], &sM[16 * k * LD + 16 * tb], l, g, x[ta][tb]);
#pragma unroll
        for (int ta = 0; ta < 2; ++ta)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) tile_put<LD>(&sM[16 * ta * LD + 32 + 16 * tb], l, g, x[ta][tb]);
        wave_order();
#pragma unroll
        for (int ta = 0; ta < 2; ++ta)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                x[ta][tb] = fz;
#pragma unroll
                for (int k = 0; k <= ta; ++k)
                    tile_mm<LD>(&sM[(32 + 16 * ta) * LD + 32 + 16 * k], &sM[16 * k * LD + 32 + 16 * tb], l, g, x[ta][tb]);
            }
#pragma unroll
        for (int ta = 0; ta < 2; ++ta)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) tile_put<LD>(&sM[(32 + 16 * ta) * LD + 16 * tb], l, g, -x[ta][tb]);
    }
    wave_order();
    bf16* dst = p.tf + ci * (int64_t)(kTriValues * WP) + 8 * lane;
    each_lower<LD>(sM, l, g, [&](int i, const f32x4& a, const f32x4& b) {
        bf16x8 o[WP];
        planes8<WP>(a, b, o);
#pragma unroll
        for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x8*>(dst + (i * WP + j) * 512) = o[j];
    });
}

template <typename IO, int N, bool BWD>
__global__ __launch_bounds__(64, 2) void delta_chunk_kernel(const DeltaParams p)
{
    __shared__ __attribute__((aligned(16))) char lds[kChunkLds];
    delta_chunk<IO, N, BWD>(p, blockIdx.x, lds);
}

template <typename IO, int N, bool BWD>
hipError_t launch_delta_chunks(const DeltaParams& p, hipStream_t stream)
{
    const int64_t blocks = delta_chunk_count(p) * p.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_chunk_kernel<IO, N, BWD>), dim3((unsigned)blocks), dim3(64), 0, stream, p);
    return hipGetLastError();
}

}  // namespace m3
