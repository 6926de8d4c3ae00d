// Gated delta rule, gradient: what needs no state's adjoint (delta_pre), the
// walk of the adjoint from the last chunk to the first (delta_back), and every
// gradient of a chunk from its state, its adjoint, U and dR (delta_grad).
//
// With P = K S0, R = beta V - sp P, U = T R, A = scale D o Q K^T (unit rows) and
// S1 = e^G_last S0 + K^T (su U), O = so (Q S0) + A U, the reverse is
//   dU  = A^T dO + su (K dS1),   dR = T^T dU
//   dS0 = e^G_last dS1 + Q^T (so dO) - K^T (sp dR)
//   dA  = dO U^T, dM = -dR U^T on A's and M's triangles, and with B1 = scale D
//   o dA, B2 = beta D o dM (k, q: unit rows, d = e^(G_last - G))
//   dq  = scale e (dO S0^T) + B1 k
//   dk  = B1^T q + (B2 + B2^T) k + d (U dS1^T) - beta e (dR S0^T)
//   dv  = beta dR,   dbeta = dR.V - e k.(dR S0^T) + sum_j D (k.k) dM
//   dG  = the products of each factor e^G with its gradient; dg_t sums dG from t
//         to the chunk's end.
// All of it in float32 (planes on matrix cores), for both io types.
#pragma once

#include "m3_delta_chunk.hpp"
#include "m3_delta_walk.hpp"

namespace m3 {

// Sum over the four lane groups (g).
template <typename T> __device__ __forceinline__ T groups_sum(T v)
{
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// E1 = A^T dO (left where dR goes) and E2 = Q^T (so dO) (where dS goes), both
// made as their transposes, so that a lane stores four neighbours.  One
// workgroup per chunk and head: wave w takes tokens 16 w .. + 15 of E1 and rows
// 16 w .. (and 16 w + 64 ..) of E2, all columns.  A comes out of Q K^T as the
// second operand.  Bound by memory: it reads a chunk's K, Q and dO and writes
// 4 (64 + N) P bytes: 56 KB a chunk and head at N = P = 64, 31 us for 2048 of
// them (3.8 TB/s).  A read from the chunk kernel instead of made here cost 12 KB
// of writes and reads each: the whole gradient took 245 for 215 us.
template <typename IO, int N, int PB> struct PreCfg {
    static constexpr int KP = DeltaPlanes<IO>::io, LQ = N + 8, LO = 32 * PB + 8;
    static constexpr int q = KP * 64 * LQ * 2, o = 2 * q, f = o + KP * 64 * LO * 2, total = f + 4 * 64 * 4;
};
template <typename IO, int N, int PB>
__global__ __launch_bounds__(256) void delta_pre_kernel(const DeltaBwdParams bp)
{
    using Cf = PreCfg<IO, N, PB>;
    const DeltaParams& p = bp.f;
    constexpr int KP = Cf::KP, WP = DeltaPlanes<IO>::wide, NT = N / 16, TI = (NT + 3) / 4, LQ = Cf::LQ, LO = Cf::LO, P = 32 * PB;
    extern __shared__ __attribute__((aligned(16))) char plds[];
    bf16 *sK = reinterpret_cast<bf16*>(plds), *sQ = reinterpret_cast<bf16*>(plds + Cf::q), *sO = reinterpret_cast<bf16*>(plds + Cf::o);
    float* sF = reinterpret_cast<float*>(plds + Cf::f);   // 1/|k|, G's two parts, 1/|q|
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bid = blockIdx.x;
    const int h = (int)(bid % p.H), bc = (int)(bid / p.H);
    int b, c;
    delta_place(p, bc, b, c);
    const DeltaRow row = delta_row(p, b);
    if ((int64_t)c * kDC >= row.len) return;
    const int64_t t0 = row.start + (int64_t)c * kDC, ci = (row.slot0 + c) * p.H + h;
    const int nv = row.len - (int64_t)c * kDC < kDC ? (int)(row.len - (int64_t)c * kDC) : kDC;
    const int hg = h / (p.H / p.G);
    const IO* qp = reinterpret_cast<const IO*>(p.q) + (t0 * p.G + hg) * N;
    const IO* kp = reinterpret_cast<const IO*>(p.k) + (t0 * p.G + hg) * N;
    const IO* op = reinterpret_cast<const IO*>(bp.dout) + (t0 * p.H + h) * P;
    const int rs = p.G * N, vs = p.H * P;
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};

    // rows past the end are zero
    auto put = [&](const IO* src, int stride, int width, bf16* dst, int ld) {
        for (int i = tid; i < 8 * width; i += 256) {
            const int t = i / (width / 8), j = i % (width / 8);
            RawRow8<IO> x;
            x.load(src + (t < nv ? t : 0) * stride + 8 * j, t < nv);
            bf16x8 o[KP];
            x.planes(o);
#pragma unroll
            for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(dst + (e * 64 + t) * ld + 8 * j) = o[e];
        }
    };
    put(kp, rs, N, sK, LQ);
    put(qp, rs, N, sQ, LQ);
    put(op, vs, P, sO, LO);
    if (tid < 192) sF[tid] = p.sc[ci * (kDScal * 64) + 320 + tid];
    __syncthreads();
    {
        const int t = 16 * w + l;
        float q2 = 0.f;
#pragma unroll
        for (int j = 0; j < N / 32; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = 0.f;
#pragma unroll
                for (int k = KP - 1; k >= 0; --k) x += (float)sQ[(k * 64 + t) * LQ + 32 * j + 8 * g + e];
                q2 += x * x;
            }
        q2 = groups_sum(q2);
        if (g == 0) sF[192 + t] = t >= nv ? 0.f : p.l2norm ? __builtin_amdgcn_rsqf(q2 + p.eps) : 1.f;
    }
    __syncthreads();

    // A's column of this lane's token j as the second operand: rows 32 kb + 8 g ..
    bf16x8 at[2][WP];
    {
        const int j = 16 * w + l;
        const float rk = sF[j], gh = sF[64 + j], gl = sF[128 + j];
        bf16x8 k8[N / 32][KP];
#pragma unroll
        for (int kn = 0; kn < N / 32; ++kn)
#pragma unroll
            for (int e = 0; e < KP; ++e) k8[kn][e] = *reinterpret_cast<const bf16x8*>(sK + (e * 64 + j) * LQ + 32 * kn + 8 * g);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int e = 0; e < WP; ++e) at[kb][e] = zero8();
            if (kb < (w >> 1)) continue;   // wave-uniform
            bf16x4 lo[WP], hi[WP];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f32x4 qk = fz;
                const int qrow = tile_row(2 * kb + s, l);
#pragma unroll
                for (int kn = 0; kn < N / 32; ++kn) {
                    bf16x8 q8[KP];
#pragma unroll
                    for (int e = 0; e < KP; ++e) q8[e] = *reinterpret_cast<const bf16x8*>(sQ + (e * 64 + qrow) * LQ + 32 * kn + 8 * g);
                    mma_planes<KP, KP, WP>(q8, k8[kn], qk);
                }
                const int i0 = 32 * kb + 8 * g + 4 * s;
                const f32x4 gh4 = *reinterpret_cast<const f32x4*>(sF + 64 + i0), gl4 = *reinterpret_cast<const f32x4*>(sF + 128 + i0);
                const f32x4 rq4 = *reinterpret_cast<const f32x4*>(sF + 192 + i0);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float D = __builtin_amdgcn_exp2f((gh4[r] - gh) + (gl4[r] - gl)) * rk;
                    qk[r] = i0 + r >= j ? p.scale * rq4[r] * D * qk[r] : 0.f;
                }
                to_planes4<WP>(qk, s == 0 ? lo : hi);
            }
#pragma unroll
            for (int e = 0; e < WP; ++e) at[kb][e] = join8(lo[e], hi[e]);
        }
    }
    // columns of Q, and so of the tokens 32 kb + 8 g ..
    auto tr8 = [&](const bf16* base, int ld, int kb, int col) {
        const bf16* s = base + (32 * kb + 8 * g + (l >> 2)) * ld + col + 4 * (l & 3);
        return join8(lds_read_tr4(s), lds_read_tr4(s + 4 * ld));
    };
    bf16x8 qt[TI][2][KP];
    float so[2][8];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int e = 0; e < KP; ++e) qt[i][kb][e] = tr8(sQ + e * 64 * LQ, LQ, kb, 16 * (w + 4 * i < NT ? w + 4 * i : 0));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = 32 * kb + 8 * g + e;
            so[kb][e] = p.scale * __builtin_amdgcn_exp2f(sF[64 + t] + sF[128 + t]) * sF[192 + t];
        }
    }
    float* e1 = bp.dR + (ci * 64 + 16 * w + l) * (int64_t)P + 4 * g;
    float* e2 = bp.dS + (ci * N + 16 * w + l) * (int64_t)P + 4 * g;
#pragma unroll
    for (int pt = 0; pt < P / 16; ++pt) {
        f32x4 a1 = fz, a2[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) a2[i] = fz;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            bf16x8 o8[KP], s8[WP];
#pragma unroll
            for (int e = 0; e < KP; ++e) o8[e] = tr8(sO + e * 64 * LO, LO, kb, 16 * pt);
            if (kb >= (w >> 1)) mma_planes<KP, WP, WP>(o8, at[kb], a1);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int j = KP - 1; j >= 0; --j) {
                    x += (float)o8[j][e];
                    y += (float)o8[j][e + 1];
                }
                bf16x2 t[WP];
                to_planes2<WP>(so[kb][e] * x, so[kb][e + 1] * y, t);
#pragma unroll
                for (int j = 0; j < WP; ++j) { s8[j][e] = t[j][0]; s8[j][e + 1] = t[j][1]; }
            }
#pragma unroll
            for (int i = 0; i < TI; ++i) mma_planes<WP, KP, WP>(s8, qt[i][kb], a2[i]);
        }
        *reinterpret_cast<f32x4*>(e1 + 16 * pt) = a1;
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT) *reinterpret_cast<f32x4*>(e2 + 64 * i * P + 16 * pt) = a2[i];
    }
}

// The adjoint's walk, for 16 columns: as the forward walk with K dS for K S,
// T^T for T and dR for d U; E1 and E2 stand in the places of dR and dS and are
// read one chunk ahead.
template <typename IO, int N>
__device__ __forceinline__ void delta_back(const DeltaBwdParams& bp, int64_t bid, char* wlds)
{
    using Cf = WalkCfg<IO, N, true>;
    constexpr int KP = Cf::KP, WP = Cf::WP, KB = Cf::KB, NT = Cf::NT, TI = Cf::TI, NBUF = Cf::NBUF;
    const DeltaParams& p = bp.f;
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int nsl = p.P / 16;
    const int64_t idx = bid >> 3;
    const int64_t unit = (idx / nsl) * 8 + (bid & 7);
    if (unit >= (int64_t)p.rows * p.H) return;
    int b, h;
    delta_unit(p, unit, b, h);
    const int64_t rec = (int64_t)b * p.H + h;
    const int p0 = (int)(idx % nsl) * 16;
    const DeltaRow row = delta_row(p, b);
    const int nch = (int)((row.len + kDC - 1) / kDC);
    const int64_t ci0 = row.slot0 * p.H + h;
    const int nlast = (int)(row.len - (int64_t)(nch - 1) * kDC);
    if (wave == 4) {
        walk_loader<IO, N, true, true>(p, wlds, p.tf, row, h, p0, nch, nlast, lane);
        return;
    }
    char* ex = wlds + Cf::ex + 16 * lane;
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};
    const int tr0 = 32 * (w >> 1) + 4 * (w & 1) + 8 * g, half = 8 * (w & 1), col = p0 + l, P = p.P;
    const int kb0 = w >> 1;   // first 32-token block of this wave's rows of T^T
    f32x4 S[TI];
    const float* hin = bp.dh_out != nullptr ? bp.dh_out + rec * (int64_t)(N * P) + col : nullptr;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][r] = hin != nullptr && w + 4 * i < NT ? hin[(tr0 + 64 * i + r) * P] : 0.f;
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            if (w + 4 * i >= NT) continue;
            bf16x4 o[WP];
            to_planes4<WP>(S[i], o);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                *reinterpret_cast<bf16x4*>(ex + Cf::s + (j * KB + 2 * i + (w >> 1)) * 1024 + half) = o[j];
        }
    };
    put_state();
    f32x4 e1, e2[TI];
    auto load_e = [&](int c) {
        const int64_t ci = ci0 + (int64_t)c * p.H;
        const float *x = bp.dR + ci * 64 * P + col, *y = bp.dS + ci * N * P + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) e1[r] = x[(tr0 + r) * P];
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r) e2[i][r] = y[(tr0 + 64 * i + r) * P];
    };
    if (nch > 0) load_e(nch - 1);
    __syncthreads();
    for (int s = 0; s < nch; ++s) {
        const int c = nch - 1 - s;
        const int64_t ci = ci0 + (int64_t)c * p.H;
        const char* buf = wlds + (s % NBUF) * Cf::buf;
        const float* f = reinterpret_cast<const float*>(buf + Cf::f) + tr0;
        const char* tb = wlds + Cf::t + (s % Cf::TB) * Cf::tsize + 16 * (16 * (l & 3) + 4 * g + (l >> 2)) + half;
        const f32x4 c1 = e1;
        f32x4 c2[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) c2[i] = e2[i];
        {
            float* sd = bp.dS + ci * N * P + col;
#pragma unroll
            for (int i = 0; i < TI; ++i)
                if (w + 4 * i < NT)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sd[(tr0 + 64 * i + r) * P] = S[i][r];
        }
        // dU = E1 + su (K dS)
        bf16x8 t8[2][WP];
        const f32x4 fp = *reinterpret_cast<const f32x4*>(f + 64), fu = *reinterpret_cast<const f32x4*>(f + 128);
        const float eL = *reinterpret_cast<const float*>(buf + Cf::f + 1024 + 4 * lane);
        f32x4 X = fz;
        {
            const int t = tile_row(w, l);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8 k8[KP], s8[WP];
#pragma unroll
                for (int j = 0; j < WP; ++j) s8[j] = *reinterpret_cast<const bf16x8*>(ex + Cf::s + (j * KB + kb) * 1024);
#pragma unroll
                for (int j = 0; j < KP; ++j)
                    k8[j] = *reinterpret_cast<const bf16x8*>(buf + Cf::k + j * (64 * N * 2) + t * (2 * N) +
                                                             16 * k_block<N>(t, 4 * kb + g));
                mma_planes<KP, WP, WP>(k8, s8, X);
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < WP; ++j) {
                    // rows of T^T: columns tile_row(w, l) of T, rows 32 kb + 8 g ..
                    // (tiles 2 kb, 2 kb + 1 of T, their column block w / 2)
                    const int k = kb < kb0 ? 1 : kb;
                    const char* s = tb + j * 1024;
                    t8[kb][j] = join8(lds_read_tr4(reinterpret_cast<const bf16*>(s + low_block(2 * k, kb0) * (WP * 1024))),
                                      lds_read_tr4(reinterpret_cast<const bf16*>(s + low_block(2 * k + 1, kb0) * (WP * 1024))));
                }
            f32x4 dU;
#pragma unroll
            for (int r = 0; r < 4; ++r) dU[r] = c1[r] + fu[r] * X[r];
            bf16x4 o[WP];
            to_planes4<WP>(dU, o);
#pragma unroll
            for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x4*>(ex + Cf::r + (2 * j + (w >> 1)) * 1024 + half) = o[j];
        }
        if (s + 1 < nch) load_e(c - 1);
        __syncthreads();
        // dR = T^T dU
        bf16x8 kt[TI][2][KP];
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int t = 32 * kb + 8 * g + (l >> 2), j4 = w + 4 * i < NT ? 4 * (2 * i + (w >> 1)) + (l & 3) : 0;
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    const char* src = buf + Cf::k + j * (64 * N * 2) + half;
                    kt[i][kb][j] = join8(lds_read_tr4(reinterpret_cast<const bf16*>(src + t * (2 * N) + 16 * k_block<N>(t, j4))),
                                         lds_read_tr4(reinterpret_cast<const bf16*>(src + (t + 4) * (2 * N) + 16 * k_block<N>(t + 4, j4))));
                }
            }
        f32x4 dR = fz;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb >= kb0) {
                bf16x8 r8[WP];
#pragma unroll
                for (int j = 0; j < WP; ++j) r8[j] = *reinterpret_cast<const bf16x8*>(ex + Cf::r + (2 * j + kb) * 1024);
                mma_planes<WP, WP, WP>(t8[kb], r8, dR);
            }
        {
            f32x4 x;
            float* rd = bp.dR + ci * 64 * P + col;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                rd[(tr0 + r) * P] = dR[r];
                x[r] = -fp[r] * dR[r];
            }
            bf16x4 o[WP];
            to_planes4<WP>(x, o);
#pragma unroll
            for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x4*>(ex + Cf::u2 + (2 * j + (w >> 1)) * 1024 + half) = o[j];
        }
        __syncthreads();
        // dS <- e^G_last dS + E2 - K^T (sp dR)
        f32x4 acc[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) acc[i] = c2[i];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            bf16x8 u8[WP], k8[TI][KP];
#pragma unroll
            for (int j = 0; j < WP; ++j) u8[j] = *reinterpret_cast<const bf16x8*>(ex + Cf::u2 + (2 * j + kb) * 1024);
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < KP; ++j) k8[i][j] = kt[i][kb][j];
            mma_tiles<TI, KP, WP, WP>(k8, u8, acc);
        }
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = eL * S[i][r] + acc[i][r];
        put_state();
        __syncthreads();
    }
    if (bp.dh_in != nullptr) {
        float* ho = bp.dh_in + rec * (int64_t)(N * P) + col;
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r) ho[(tr0 + 64 * i + r) * P] = S[i][r];
    }
}

// Both walks of the gradient: neither needs the other, and each alone waits
// for its own chain most of the time.  All workgroups of one, then of the
// other, so that a CU gets one of each.  79 us at 256 slices, 32 chunks, N = P =
// 64 (107 as two launches), about 156 KB of memory traffic a chunk and head
// (4.1 TB/s).
template <typename IO, int N>
__global__ __launch_bounds__(320) void delta_walks_kernel(const DeltaBwdParams bp)
{
    extern __shared__ __attribute__((aligned(16))) char wlds[];
    const unsigned n = gridDim.x / 2;   // a multiple of 8: the XCDs of both halves agree
    if (blockIdx.x < n) delta_back<IO, N>(bp, blockIdx.x, wlds);
    else delta_walk<IO, N, true>(bp.f, bp.S, bp.U, blockIdx.x - n, wlds);
}

template <typename IO, int N, int PB> struct GradCfg {
    static constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide, P = 32 * PB;
    static constexpr int LK = N + 8, LP = P + 8, LB = 68;
    // bytes: K, Q | one after the other: S0 and dS1 tiles (twice), U, B1 and B2 | the rest
    static constexpr int q = KP * 64 * LK * 2, x = 2 * q, tile = WP * 16 * LP * 2, xs = 4 * tile, xu = WP * 64 * LP * 2,
                         xb = 2 * 64 * LB * 4;
    static constexpr int xmax = xs > xu ? (xs > xb ? xs : xb) : (xu > xb ? xu : xb);
    static constexpr int f = x + xmax, total = f + (9 * 64 + 64 + 4) * 4 + (4 * 64 + 64) * 8;
    static_assert(f % 8 == 0, "float64 values behind 9 rows of 64 factors");
};

// Every gradient of one chunk of one head.  Wave w has tokens 16 w .. + 15:
// every product is made as its transpose, so that a lane has one token (l) and
// its row's factors and sums are scalars of the lane, and results leave as four
// neighbours.  The rows of dO, dR and U are second operands as they lie in
// memory; S0 and dS1 go through LDS in tiles of 16 rows, split once for all
// four waves, the next tile's loads in flight; then U takes that place, then
// B1 and B2, whose columns dk needs.  Bound by memory: a chunk's two states, U,
// dR and its rows come in once, 64 KB of gradients go out; 144 KB a chunk and
// head at N = P = 64, 95 us for 2048 of them (3.1 TB/s) with two workgroups to a
// CU.  With a lane for four rows instead of one (products not transposed) the
// factors, sums and stores were four times as many: 193 us.
template <typename IO, int N, int PB>
__global__ __launch_bounds__(256, PB <= 2 ? 2 : 1) void delta_grad_kernel(const DeltaBwdParams bp)
{
    using Cf = GradCfg<IO, N, PB>;
    const DeltaParams& p = bp.f;
    constexpr int KP = Cf::KP, WP = Cf::WP, NT = N / 16, LK = Cf::LK, LP = Cf::LP, LB = Cf::LB, P = Cf::P;
    extern __shared__ __attribute__((aligned(16))) char glds[];
    bf16* sK = reinterpret_cast<bf16*>(glds);
    bf16* sQ = reinterpret_cast<bf16*>(glds + Cf::q);
    bf16* sX = reinterpret_cast<bf16*>(glds + Cf::x);
    float* sB1 = reinterpret_cast<float*>(glds + Cf::x);
    float* sB2 = sB1 + 64 * LB;
    float* sF = reinterpret_cast<float*>(glds + Cf::f);   // [8][64] factors, [64] 1/|q|
    float* sRq = sF + 8 * 64;
    double* sCol = reinterpret_cast<double*>(sRq + 64);   // [4][64] column sums of each wave's rows
    double* sG = sCol + 256;   // [64] dG but for the column sums and the total
    float* sUs = reinterpret_cast<float*>(sG + 64);       // [64] what the factor d adds to G_last and takes from G
    float* sTot = sUs + 64;    // [4] each wave's share of <S0, dS1>
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bid = blockIdx.x;
    const int h = (int)(bid % p.H), bc = (int)(bid / p.H);
    int b, c;
    delta_place(p, bc, b, c);
    const DeltaRow row = delta_row(p, b);
    if ((int64_t)c * kDC >= row.len) return;
    const int64_t t0 = row.start + (int64_t)c * kDC, ci = (row.slot0 + c) * p.H + h;
    const int nv = row.len - (int64_t)c * kDC < kDC ? (int)(row.len - (int64_t)c * kDC) : kDC;
    const int hg = h / (p.H / p.G);
    const IO* qp = reinterpret_cast<const IO*>(p.q) + (t0 * p.G + hg) * N;
    const IO* kp = reinterpret_cast<const IO*>(p.k) + (t0 * p.G + hg) * N;
    const IO* op = reinterpret_cast<const IO*>(bp.dout) + (t0 * p.H + h) * P;
    const IO* vp = reinterpret_cast<const IO*>(p.v) + (t0 * p.H + h) * P;
    const int rs = p.G * N, vs = p.H * P;
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};

    // the tiles of S0 and dS1: this thread's four values of each, SI times
    constexpr int SI = (16 * P / 4 + 255) / 256;
    const float* Sb = bp.S + ci * N * (int64_t)P;
    const float* Db = bp.dS + ci * N * (int64_t)P;
    f32x4 sr[SI], dr[SI];
    auto load_tile = [&](int nt) {
#pragma unroll
        for (int i = 0; i < SI; ++i) {
            int j = tid + 256 * i;
            if (16 * P / 4 % 256 != 0 && j >= 16 * P / 4) j = 0;   // (stored by thread 0 alone)
            sr[i] = *reinterpret_cast<const f32x4*>(Sb + nt * 16 * P + 4 * j);
            dr[i] = *reinterpret_cast<const f32x4*>(Db + nt * 16 * P + 4 * j);
        }
    };
    float tot = 0.f;
    auto put_tile = [&](int nt) {
        bf16* s = sX + (nt & 1) * (Cf::tile);   // (two tiles of `tile` bytes each)
#pragma unroll
        for (int i = 0; i < SI; ++i) {
            const int j = tid + 256 * i;
            if (16 * P / 4 % 256 != 0 && j >= 16 * P / 4) continue;
            const int r = j / (P / 4), x = j % (P / 4);
            bf16x4 o[WP];
            to_planes4<WP>(sr[i], o);
#pragma unroll
            for (int e = 0; e < WP; ++e) *reinterpret_cast<bf16x4*>(s + (e * 16 + r) * LP + 4 * x) = o[e];
            to_planes4<WP>(dr[i], o);
#pragma unroll
            for (int e = 0; e < WP; ++e) *reinterpret_cast<bf16x4*>(s + Cf::tile / 2 + (e * 16 + r) * LP + 4 * x) = o[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) tot += sr[i][e] * dr[i][e];
        }
    };
    load_tile(0);

    // second operands: rows of dO, dR, U; dv, and dR.V for dbeta
    const int irow = 16 * w + l;   // this lane's token
    const bool real = irow < nv;
    bf16x8 o8[PB][KP], r8[PB][WP], u8[PB][WP];
    float drv = 0.f;
    const float* Ub = bp.U + ci * 64 * (int64_t)P;
    const float* Rb = bp.dR + ci * 64 * (int64_t)P;
    const float* sc = p.sc + ci * (kDScal * 64);
    const float beta = sc[irow];
    {
        RawRow8<IO> x[PB], v[PB];
        RawRow8<float> r[PB], u[PB];
#pragma unroll
        for (int kb = 0; kb < PB; ++kb) {
            const int pc = 32 * kb + 8 * g;
            x[kb].load(op + (real ? irow : 0) * vs + pc, real);
            v[kb].load(vp + (real ? irow : 0) * vs + pc, real);
            r[kb].load(Rb + irow * P + pc, true);
            u[kb].load(Ub + irow * P + pc, true);
        }
        // K, Q to LDS, rows past the end zero
        for (int i = tid; i < 64 * N / 8; i += 256) {
            const int t = i / (N / 8), j = i % (N / 8);
            RawRow8<IO> y, z;
            y.load(kp + (t < nv ? t : 0) * rs + 8 * j, t < nv);
            z.load(qp + (t < nv ? t : 0) * rs + 8 * j, t < nv);
            bf16x8 o[KP];
            y.planes(o);
#pragma unroll
            for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sK + (e * 64 + t) * LK + 8 * j) = o[e];
            z.planes(o);
#pragma unroll
            for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sQ + (e * 64 + t) * LK + 8 * j) = o[e];
        }
        for (int i = tid; i < kDScal * 64; i += 256) sF[i] = sc[i];
        put_tile(0);
#pragma unroll
        for (int kb = 0; kb < PB; ++kb) {
            x[kb].planes(o8[kb]);
            r[kb].planes(r8[kb]);
            u[kb].planes(u8[kb]);
            f32x4 d0, d1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                drv += r[kb].get(e) * v[kb].get(e);
                if (e < 4) d0[e] = beta * r[kb].get(e);
                else d1[e - 4] = beta * r[kb].get(e);
            }
            if (real) {
                float* dv = bp.dv + ((t0 + irow) * p.H + h) * P + 32 * kb + 8 * g;
                *reinterpret_cast<f32x4*>(dv) = d0;
                *reinterpret_cast<f32x4*>(dv + 4) = d1;
            }
        }
    }
    drv = groups_sum(drv);
    __syncthreads();

    // this token's factors
    float q2 = 0.f;
#pragma unroll
    for (int j = 0; j < N / 32; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x = 0.f;
#pragma unroll
            for (int k = KP - 1; k >= 0; --k) x += (float)sQ[(k * 64 + irow) * LK + 32 * j + 8 * g + e];
            q2 += x * x;
        }
    q2 = groups_sum(q2);
    const float rq = !real ? 0.f : p.l2norm ? __builtin_amdgcn_rsqf(q2 + p.eps) : 1.f;
    if (g == 0) sRq[irow] = rq;   // (read after the next barriers)
    const float rk = sF[320 + irow], gh = sF[384 + irow], gl = sF[448 + irow];
    const float eG = __builtin_amdgcn_exp2f(gh + gl);
    const float dG = __builtin_amdgcn_exp2f((sF[384 + 63] - gh) + (sF[448 + 63] - gl));

    // dO S0^T, dR S0^T, U dS1^T: rows 16 nt + 4 g + r of their transposes
    f32x4 accq[NT], acck[NT];
    float qs = 0.f, ks = 0.f, us = 0.f;
    // four values of this token's unit row, columns 16 nt + 4 g ..
    auto row4 = [&](const bf16* s, int nt, float scale) {
        f32x4 x = fz;
#pragma unroll
        for (int e = KP - 1; e >= 0; --e) {
            const bf16x4 y = *reinterpret_cast<const bf16x4*>(s + (e * 64 + irow) * LK + 16 * nt + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] += (float)y[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] *= scale;
        return x;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (nt + 1 < NT) load_tile(nt + 1);
        const bf16* s = sX + (nt & 1) * Cf::tile + l * LP + 8 * g;
        f32x4 w1 = fz, w2 = fz, w3 = fz;
#pragma unroll
        for (int kb = 0; kb < PB; ++kb) {
            bf16x8 s8[WP], d8[WP];
#pragma unroll
            for (int e = 0; e < WP; ++e) {
                s8[e] = *reinterpret_cast<const bf16x8*>(s + e * 16 * LP + 32 * kb);
                d8[e] = *reinterpret_cast<const bf16x8*>(s + Cf::tile / 2 + e * 16 * LP + 32 * kb);
            }
            mma_planes<WP, KP, WP>(s8, o8[kb], w1);
            mma_planes<WP, WP, WP>(s8, r8[kb], w2);
            mma_planes<WP, WP, WP>(d8, u8[kb], w3);
        }
        const f32x4 qv = row4(sQ, nt, rq), kv = row4(sK, nt, rk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float x = p.scale * eG * w1[r], y = eG * w2[r], z = dG * w3[r];
            qs += qv[r] * x;
            ks += kv[r] * y;
            us += kv[r] * z;
            accq[nt][r] = x;
            acck[nt][r] = z - beta * y;
        }
        if (nt + 1 < NT) put_tile(nt + 1);
        __syncthreads();
    }
    qs = groups_sum(qs);
    ks = groups_sum(ks);
    us = groups_sum(us);
    tot = groups_sum(lane_group_sum<16>(tot));
    if (lane == 0) sTot[w] = tot;

    // U's planes where the tiles were
#pragma unroll
    for (int kb = 0; kb < PB; ++kb)
#pragma unroll
        for (int e = 0; e < WP; ++e) *reinterpret_cast<bf16x8*>(sX + (e * 64 + irow) * LP + 32 * kb + 8 * g) = u8[kb][e];
    __syncthreads();

    // B1, B2 (this token's row, keys 16 ct + 4 g + r), the row and column sums
    // of Z = B1 (q.k) + B2 (k.k), and the M part of dbeta.  A key's column takes
    // from dg what the tokens' rows gave, so both are summed in float64: dg's error
    // was 3.3e-7 with float32 sums and is 1.7e-7, for 1% of the call.
    double zrow = 0.;
    float mrow = 0.f;
    f32x4 v1[4], v2[4];
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        double zc[4] = {0., 0., 0., 0.};
        v1[ct] = fz;
        v2[ct] = fz;
        if (ct <= w) {   // wave-uniform
            f32x4 qk = fz, kk = fz, dA = fz, dM = fz;
#pragma unroll
            for (int kb = 0; kb < N / 32; ++kb) {
                bf16x8 a[KP], q[KP], j[KP];
#pragma unroll
                for (int e = 0; e < KP; ++e) {
                    a[e] = *reinterpret_cast<const bf16x8*>(sK + (e * 64 + irow) * LK + 32 * kb + 8 * g);
                    q[e] = *reinterpret_cast<const bf16x8*>(sQ + (e * 64 + irow) * LK + 32 * kb + 8 * g);
                    j[e] = *reinterpret_cast<const bf16x8*>(sK + (e * 64 + 16 * ct + l) * LK + 32 * kb + 8 * g);
                }
                mma_planes<KP, KP, WP>(j, a, kk);
                mma_planes<KP, KP, WP>(j, q, qk);
            }
#pragma unroll
            for (int kb = 0; kb < PB; ++kb) {
                bf16x8 j[WP];
#pragma unroll
                for (int e = 0; e < WP; ++e)
                    j[e] = *reinterpret_cast<const bf16x8*>(sX + (e * 64 + 16 * ct + l) * LP + 32 * kb + 8 * g);
                mma_planes<WP, KP, WP>(j, o8[kb], dA);
                mma_planes<WP, WP, WP>(j, r8[kb], dM);
            }
            const int j0 = 16 * ct + 4 * g;
            const f32x4 rk4 = *reinterpret_cast<const f32x4*>(sF + 320 + j0);
            const f32x4 gh4 = *reinterpret_cast<const f32x4*>(sF + 384 + j0);
            const f32x4 gl4 = *reinterpret_cast<const f32x4*>(sF + 448 + j0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float D = __builtin_amdgcn_exp2f((gh - gh4[r]) + (gl - gl4[r]));
                if (ct == w && 4 * g + r > l) D = 0.f;
                const float dm = (ct == w && 4 * g + r >= l) ? 0.f : -D * dM[r];
                const float b1 = p.scale * D * dA[r], kn = rk * rk4[r] * kk[r], b2 = beta * dm;
                const float z = b1 * (rq * rk4[r] * qk[r]) + b2 * kn;
                zrow += z;
                mrow += dm * kn;
                zc[r] = z;
                v1[ct][r] = b1;
                v2[ct][r] = b2;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            zc[r] = lane_group_sum_d(zc[r]);
            if (l == 0) sCol[w * 64 + 16 * ct + 4 * g + r] = zc[r];
        }
    }
    zrow = groups_sum(zrow);
    mrow = groups_sum(mrow);
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        *reinterpret_cast<f32x4*>(sB1 + irow * LB + 16 * ct + 4 * g) = v1[ct];
        *reinterpret_cast<f32x4*>(sB2 + irow * LB + 16 * ct + 4 * g) = v2[ct];
    }
    // dbeta and dG of this token
    if (g == 0) {
        sG[irow] = (double)qs - (double)beta * ks + zrow - us;
        sUs[irow] = us;
        if (real) bp.dbeta[(t0 + irow) * p.H + h] = drv - ks + mrow;
    }
    __syncthreads();

    // second operands from B1 (rows: dq; columns: dk) and B2 + B2^T (dk), with
    // the unit factors of the first operands' rows; zero off their triangles
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        bf16x8 b1[WP], b1t[WP], b2[WP];
        const int j0 = 32 * kb + 8 * g;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float x[2], y[2], z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = j0 + e + i;
                const float rkj = sF[320 + j];
                x[i] = sB1[irow * LB + j] * rkj;
                y[i] = sB1[j * LB + irow] * sRq[j];
                z[i] = (sB2[irow * LB + j] + sB2[j * LB + irow]) * rkj;
            }
            bf16x2 t[WP];
            to_planes2<WP>(x[0], x[1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b1[i][e] = t[i][0]; b1[i][e + 1] = t[i][1]; }
            to_planes2<WP>(y[0], y[1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b1t[i][e] = t[i][0]; b1t[i][e + 1] = t[i][1]; }
            to_planes2<WP>(z[0], z[1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b2[i][e] = t[i][0]; b2[i][e + 1] = t[i][1]; }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            bf16x8 kt[KP], qt[KP];
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                const int at = (e * 64 + j0 + (l >> 2)) * LK + 16 * nt + 4 * (l & 3);
                kt[e] = join8(lds_read_tr4(sK + at), lds_read_tr4(sK + at + 4 * LK));
                qt[e] = join8(lds_read_tr4(sQ + at), lds_read_tr4(sQ + at + 4 * LK));
            }
            mma_planes<KP, WP, WP>(kt, b1, accq[nt]);
            mma_planes<KP, WP, WP>(qt, b1t, acck[nt]);
            mma_planes<KP, WP, WP>(kt, b2, acck[nt]);
        }
    }

    // dq, dk through the unit rows: r (d - x (x.d))
    float qd = 0.f, kd = 0.f;
    if (p.l2norm) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const f32x4 qv = row4(sQ, nt, rq), kv = row4(sK, nt, rk);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                qd += qv[r] * accq[nt][r];
                kd += kv[r] * acck[nt][r];
            }
        }
        qd = groups_sum(qd);
        kd = groups_sum(kd);
    }
    if (real) {
        const int64_t at = ((t0 + irow) * p.H + h) * N + 4 * g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            f32x4 dq = accq[nt], dk = acck[nt];
            if (p.l2norm) {
                const f32x4 qv = row4(sQ, nt, rq), kv = row4(sK, nt, rk);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dq[r] = rq * (dq[r] - qv[r] * qd);
                    dk[r] = rk * (dk[r] - kv[r] * kd);
                }
            }
            *reinterpret_cast<f32x4*>(bp.dqe + at + 16 * nt) = dq;
            *reinterpret_cast<f32x4*>(bp.dke + at + 16 * nt) = dk;
        }
    }
    if (w == 0) {
        double x = sG[lane] - (sCol[lane] + sCol[64 + lane] + sCol[128 + lane] + sCol[192 + lane]);
        const double u = wave_inclusive_sum_d((double)sUs[lane]);
        if (lane == 63) x += u + (double)sF[256] * ((double)sTot[0] + sTot[1] + sTot[2] + sTot[3]);
        const double s = wave_inclusive_sum_d(x);
        const double all = __shfl(s, 63);
        if (lane < nv) bp.dg[(t0 + lane) * p.H + h] = (float)(all - s + x);
    }
}

// dq and dk of a group of heads: the sum over its heads, in their order (zeros
// where it has none).
static __global__ __launch_bounds__(256) void delta_heads_kernel(const float* eq, const float* ek, float* oq, float* ok,
                                                                  int64_t tokens, int H, int G, int N)
{
    const float* e = blockIdx.y ? ek : eq;
    float* out = blockIdx.y ? ok : oq;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= tokens * G * N) return;
    const int64_t t = i / ((int64_t)G * N);
    const int j = (int)(i - t * G * N), gi = j / N, reach = H / G;
    const float* src = e + (t * H + (int64_t)gi * reach) * N + (j - gi * N);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < reach; ++k) s += *reinterpret_cast<const f32x4*>(src + (int64_t)k * N);
    *reinterpret_cast<f32x4*>(out + i) = s;
}

// Packed sequences: zeros where no sequence's tokens lie (before the first,
// behind the last), and where one is longer than max_seqlen says.
struct DeltaRest {
    float* a[5];
    int n[5];   // values per token
};
static __global__ __launch_bounds__(256) void delta_rest_kernel(const DeltaParams p, const DeltaRest r)
{
    const int i = blockIdx.x;   // the gap before row i
    int64_t lo = 0, hi = p.L;
    if (i > 0) {
        const DeltaRow x = delta_row(p, i - 1);
        lo = x.start + x.len;
    }
    if (i < p.rows) hi = delta_row(p, i).start;
    if (lo >= hi) return;
    for (int k = 0; k < 5; ++k) {
        const int64_t n = (hi - lo) * r.n[k];
        for (int64_t j = (int64_t)blockIdx.y * 256 + threadIdx.x; j < n; j += (int64_t)gridDim.y * 256) r.a[k][lo * r.n[k] + j] = 0.f;
    }
}

template <typename IO, int N, int PB>
hipError_t launch_delta_pre(const DeltaBwdParams& bp, hipStream_t stream)
{
    auto* const kern = &delta_pre_kernel<IO, N, PB>;
    constexpr size_t lds = PreCfg<IO, N, PB>::total;
    static_assert(lds <= 160 * 1024, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    const hipError_t attr = delta_allow_lds(kern, lds, done);
    if (attr != hipSuccess) return attr;
    const int64_t blocks = delta_chunk_count(bp.f) * bp.f.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), lds, stream, bp);
    return hipGetLastError();
}

template <typename IO, int N, int PB>
hipError_t launch_delta_grad(const DeltaBwdParams& bp, hipStream_t stream)
{
    auto* const kern = &delta_grad_kernel<IO, N, PB>;
    constexpr size_t lds = GradCfg<IO, N, PB>::total;
    static_assert(lds <= 160 * 1024, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    const hipError_t attr = delta_allow_lds(kern, lds, done);
    if (attr != hipSuccess) return attr;
    const int64_t blocks = delta_chunk_count(bp.f) * bp.f.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), lds, stream, bp);
    return hipGetLastError();
}

template <typename IO, int N>
hipError_t bwd_n(const DeltaBwdParams& bp, hipStream_t stream)
{
    const DeltaParams& p = bp.f;
    hipError_t e = launch_delta_chunks<IO, N, true>(p, stream);
    if (e != hipSuccess) return e;
    switch (p.P) {
    case 32: e = launch_delta_pre<IO, N, 1>(bp, stream); break;
    case 64: e = launch_delta_pre<IO, N, 2>(bp, stream); break;
    case 96: e = launch_delta_pre<IO, N, 3>(bp, stream); break;
    default: e = launch_delta_pre<IO, N, 4>(bp, stream);
    }
    if (e != hipSuccess) return e;
    if (p.rows > 0 && p.H > 0) {
        using Cf = WalkCfg<IO, N, true>;
        auto* const walks = &delta_walks_kernel<IO, N>;
        static_assert(Cf::total <= 160 * 1024, "a workgroup's LDS");
        static std::atomic<uint64_t> done{0};
        if ((e = delta_allow_lds(walks, Cf::total, done)) != hipSuccess) return e;
        const int64_t n = ((int64_t)p.rows * p.H + 7) / 8 * 8 * (p.P / 16);
        const size_t lds = Cf::total;
        hipLaunchKernelGGL(walks, dim3((unsigned)(2 * n)), dim3(64 * Cf::waves), lds, stream, bp);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    switch (p.P) {
    case 32: e = launch_delta_grad<IO, N, 1>(bp, stream); break;
    case 64: e = launch_delta_grad<IO, N, 2>(bp, stream); break;
    case 96: e = launch_delta_grad<IO, N, 3>(bp, stream); break;
    default: e = launch_delta_grad<IO, N, 4>(bp, stream);
    }
    if (e != hipSuccess) return e;
    const int64_t tokens = p.cu != nullptr ? p.L : p.rows * p.L;
    if (p.cu != nullptr && p.L > 0 && p.H > 0) {
        const DeltaRest r = {{bp.dqe, bp.dke, bp.dv, bp.dg, bp.dbeta}, {p.H * p.N, p.H * p.N, p.H * p.P, p.H, p.H}};
        hipLaunchKernelGGL(delta_rest_kernel, dim3(p.rows + 1, 16), dim3(256), 0, stream, p, r);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.G != p.H && tokens > 0) {
        const int64_t n = (tokens * p.G * p.N / 4 + 255) / 256;
        hipLaunchKernelGGL(delta_heads_kernel, dim3((unsigned)n, 2), dim3(256), 0, stream, bp.dqe, bp.dke, bp.dq, bp.dk, tokens,
                           p.H, p.G, p.N);
        e = hipGetLastError();
    }
    return e;
}

template <typename IO>
hipError_t launch_delta_bwd_io(const DeltaBwdParams& bp, hipStream_t stream)
{
    switch (bp.f.N) {
    case 32: return bwd_n<IO, 32>(bp, stream);
    case 64: return bwd_n<IO, 64>(bp, stream);
    default: return bwd_n<IO, 128>(bp, stream);
    }
}

}  // namespace m3
