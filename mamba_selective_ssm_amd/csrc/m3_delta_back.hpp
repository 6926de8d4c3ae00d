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

// E1 = A^T dO (left where dR goes) and E2 = Q^T (so dO) (where dS goes).  One
// workgroup per chunk and head: wave w takes row tile w of E1 and the state
// tiles w, w + 4 of E2, all columns.  Bound by what it writes (4 (64 + N) P
// bytes a chunk).
template <typename IO, int N>
__global__ __launch_bounds__(256) void delta_pre_kernel(const DeltaBwdParams bp)
{
    const DeltaParams& p = bp.f;
    constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide, NT = N / 16, TI = (NT + 3) / 4, LQ = N + 8, LO = 136;
    __shared__ __attribute__((aligned(16))) bf16 sQ[KP * 64 * LQ];
    __shared__ __attribute__((aligned(16))) bf16 sO[KP * 64 * LO];
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bid = blockIdx.x;
    const int h = (int)(bid % p.H), bc = (int)(bid / p.H);
    const int c = bc % p.nc, b = bc / p.nc;
    const DeltaRow row = delta_row(p, b);
    if ((int64_t)c * kDC >= row.len) return;
    const int64_t t0 = row.start + (int64_t)c * kDC, ci = (row.slot0 + c) * p.H + h;
    const int nv = row.len - (int64_t)c * kDC < kDC ? (int)(row.len - (int64_t)c * kDC) : kDC;
    const IO* qp = reinterpret_cast<const IO*>(p.q) + (t0 * p.G + h / (p.H / p.G)) * N;
    const IO* op = reinterpret_cast<const IO*>(bp.dout) + (t0 * p.H + h) * p.P;
    const int rs = p.G * N, vs = p.H * p.P, P = p.P;

    // rows past the end are zero
    for (int i = tid; i < 64 * N / 8; i += 256) {
        const int t = i / (N / 8), j = i % (N / 8);
        RawRow8<IO> x;
        x.load(qp + (t < nv ? t : 0) * rs + 8 * j, t < nv);
        bf16x8 o[KP];
        x.planes(o);
#pragma unroll
        for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sQ + (e * 64 + t) * LQ + 8 * j) = o[e];
    }
    for (int i = tid; i < 8 * P; i += 256) {
        const int t = i / (P / 8), j = i % (P / 8);
        RawRow8<IO> x;
        x.load(op + (t < nv ? t : 0) * vs + 8 * j, t < nv);
        bf16x8 o[KP];
        x.planes(o);
#pragma unroll
        for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sO + (e * 64 + t) * LO + 8 * j) = o[e];
    }
    // A^T's rows of this wave: 32-token blocks w / 2 .. 1
    bf16x8 at[2][WP];
    const bf16* ap = bp.atf + ci * (kTriBlocks * WP * 512) + lane * 8;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < WP; ++j)
            at[kb][j] = *reinterpret_cast<const bf16x8*>(ap + (up_block(w, kb < (w >> 1) ? 1 : kb) * WP + j) * 512);
    const float* f = p.sc + ci * (kDScal * 64) + 192;
    float so[2][8];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < 8; ++e) so[kb][e] = f[32 * kb + 8 * g + e];
    __syncthreads();
    // Q^T's rows of this wave
    bf16x8 qt[TI][2][KP];
    auto tr8 = [&](const bf16* base, int ld, int kb, int col) {
        const bf16* s = base + (32 * kb + 8 * g + (l >> 2)) * ld + col;
        return join8(lds_read_tr4(s), lds_read_tr4(s + 4 * ld));
    };
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                const int ti = w + 4 * i < NT ? w + 4 * i : 0;
                qt[i][kb][e] = tr8(sQ + e * 64 * LQ, LQ, kb, 32 * (ti >> 1) + 8 * (l & 3) + 4 * (ti & 1));
            }
    const int tr0 = 32 * (w >> 1) + 4 * (w & 1) + 8 * g;
    float* e1 = bp.dR + ci * 64 * (int64_t)P;
    float* e2 = bp.dS + ci * N * (int64_t)P;
    for (int pt = 0; pt < P / 16; ++pt) {
        f32x4 a1 = {0.f, 0.f, 0.f, 0.f}, a2[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) a2[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            bf16x8 o8[KP], s8[WP];
#pragma unroll
            for (int e = 0; e < KP; ++e) o8[e] = tr8(sO + e * 64 * LO, LO, kb, 16 * pt + 4 * (l & 3));
            if (kb >= (w >> 1)) mma_planes<WP, KP, WP>(at[kb], o8, a1);
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
            for (int i = 0; i < TI; ++i) mma_planes<KP, WP, WP>(qt[i][kb], s8, a2[i]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) e1[(tr0 + r) * P + 16 * pt + l] = a1[r];
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r) e2[(tr0 + 64 * i + r) * P + 16 * pt + l] = a2[i][r];
    }
}

// The adjoint's walk, for 16 columns: as the forward walk with K dS for K S,
// T^T for T and dR for d U; E1 and E2 stand in the places of dR and dS and are
// read one chunk ahead.
template <typename IO, int N>
__global__ __launch_bounds__(320) void delta_back_kernel(const DeltaBwdParams bp)
{
    using Cf = WalkCfg<IO, N, 1>;
    constexpr int KP = Cf::KP, WP = Cf::WP, KB = Cf::KB, NT = Cf::NT, TI = Cf::TI, NBUF = Cf::NBUF;
    const DeltaParams& p = bp.f;
    extern __shared__ __attribute__((aligned(16))) char wlds[];
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int nsl = p.P / 16;
    const int64_t idx = blockIdx.x >> 3;
    const int64_t unit = (idx / nsl) * 8 + (blockIdx.x & 7);
    if (unit >= (int64_t)p.rows * p.H) return;
    int64_t b64, h64;
    split_bh(unit, p.H, b64, h64);
    const int b = (int)b64, h = (int)h64, p0 = (int)(idx % nsl) * 16;
    const DeltaRow row = delta_row(p, b);
    const int nch = (int)((row.len + kDC - 1) / kDC);
    const int64_t ci0 = row.slot0 * p.H + h;
    const int nlast = (int)(row.len - (int64_t)(nch - 1) * kDC);
    if (wave == 4) {
        walk_loader<IO, N, 1, true>(p, wlds, bp.ttf, row, h, p0, nch, nlast, lane);
        return;
    }
    char* ex = wlds + Cf::ex + 16 * lane;
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};
    const int tr0 = 32 * (w >> 1) + 4 * (w & 1) + 8 * g, half = 8 * (w & 1), col = p0 + l, P = p.P;
    const int kb0 = w >> 1;   // first 32-token block of this wave's rows of T^T
    f32x4 S[TI];
    const float* hin = bp.dh_out != nullptr ? bp.dh_out + unit * (int64_t)(N * P) + col : nullptr;
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
        const char* tb = wlds + Cf::t + (s % Cf::TB) * Cf::tsize + 16 * lane;
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
                for (int j = 0; j < WP; ++j)
                    t8[kb][j] = *reinterpret_cast<const bf16x8*>(tb + (up_block(w, kb < kb0 ? 1 : kb) * WP + j) * 1024);
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
        float* ho = bp.dh_in + unit * (int64_t)(N * P) + col;
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r) ho[(tr0 + 64 * i + r) * P] = S[i][r];
    }
}

// Sum over the 16 lanes of one row tile's columns, over the four row groups.
__device__ __forceinline__ float lanes_sum(float v) { return lane_group_sum<16>(v); }
__device__ __forceinline__ float groups_sum(float v)
{
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// Every gradient of one chunk of one head.  Wave w has tokens 16 w .. + 15, as
// rows of every product.  The rows of dO, dR and U are first operands as they
// lie in memory, S0 and dS1 second operands (each value split where it is
// used); B1 and B2 go through LDS once, because dk needs their columns.
template <typename IO, int N, int PB>
__global__ __launch_bounds__(256) void delta_grad_kernel(const DeltaBwdParams bp)
{
    const DeltaParams& p = bp.f;
    constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide, NT = N / 16, LK = N + 8, LB = 68, P = 32 * PB;
    extern __shared__ __attribute__((aligned(16))) char glds[];
    bf16* sK = reinterpret_cast<bf16*>(glds);
    bf16* sQ = sK + KP * 64 * LK;
    float* sB1 = reinterpret_cast<float*>(sQ + KP * 64 * LK);
    float* sB2 = sB1 + 64 * LB;
    float* sCol = sB2 + 64 * LB;    // [4][64] column sums of each wave's rows
    float* sG = sCol + 256;         // [64] dG but for the column sums and the total
    float* sUs = sG + 64;           // [64] what the factor d adds to G_last and takes from G
    float* sDb = sUs + 64;          // [64] dR.V
    float* sF = sDb + 64;           // [8][64] factors and [64] 1/|q|
    float* sTot = sF + 9 * 64;      // [4] each wave's share of <S0, dS1>
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bid = blockIdx.x;
    const int h = (int)(bid % p.H), bc = (int)(bid / p.H);
    const int c = bc % p.nc, b = bc / p.nc;
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

    // K, Q to LDS, rows past the end zero
    for (int i = tid; i < 64 * N / 8; i += 256) {
        const int t = i / (N / 8), j = i % (N / 8);
        RawRow8<IO> x, y;
        x.load(kp + (t < nv ? t : 0) * rs + 8 * j, t < nv);
        y.load(qp + (t < nv ? t : 0) * rs + 8 * j, t < nv);
        bf16x8 o[KP];
        x.planes(o);
#pragma unroll
        for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sK + (e * 64 + t) * LK + 8 * j) = o[e];
        y.planes(o);
#pragma unroll
        for (int e = 0; e < KP; ++e) *reinterpret_cast<bf16x8*>(sQ + (e * 64 + t) * LK + 8 * j) = o[e];
    }
    const float* sc = p.sc + ci * (kDScal * 64);
    for (int i = tid; i < kDScal * 64; i += 256) sF[i] = sc[i];
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};

    // first operands: rows of dO, dR, U; dv, and dR.V for dbeta
    const int irow = 16 * w + l, drow = 16 * w + 4 * g;
    const bool real = irow < nv;
    bf16x8 o8[PB][KP], r8[PB][WP], u8[PB][WP];
    float drv = 0.f;
    const float* Ub = bp.U + ci * 64 * (int64_t)P;
    const float* Rb = bp.dR + ci * 64 * (int64_t)P;
    const float bi = sc[irow];
#pragma unroll
    for (int kb = 0; kb < PB; ++kb) {
        const int pc = 32 * kb + 8 * g;
        RawRow8<IO> x, v;
        RawRow8<float> r, u;
        x.load(op + (real ? irow : 0) * vs + pc, real);
        v.load(vp + (real ? irow : 0) * vs + pc, real);
        r.load(Rb + irow * P + pc, true);
        u.load(Ub + irow * P + pc, true);
        x.planes(o8[kb]);
        r.planes(r8[kb]);
        u.planes(u8[kb]);
        f32x4 d0, d1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            drv += r.get(e) * v.get(e);
            if (e < 4) d0[e] = bi * r.get(e);
            else d1[e - 4] = bi * r.get(e);
        }
        if (real) {
            float* dv = bp.dv + ((t0 + irow) * p.H + h) * P + pc;
            *reinterpret_cast<f32x4*>(dv) = d0;
            *reinterpret_cast<f32x4*>(dv + 4) = d1;
        }
    }
    drv = groups_sum(drv);   // of token irow
    if (g == 0) sDb[irow] = drv;
    __syncthreads();

    // 1/|q| of the wave's tokens
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
    float* sRq = sF + kDScal * 64;
    if (g == 0) sRq[irow] = !real ? 0.f : p.l2norm ? __builtin_amdgcn_rsqf(q2 + p.eps) : 1.f;
    wave_order();
    const f32x4 beta4 = *reinterpret_cast<const f32x4*>(sF + drow);
    const f32x4 rk4 = *reinterpret_cast<const f32x4*>(sF + 320 + drow), rq4 = *reinterpret_cast<const f32x4*>(sRq + drow);
    const f32x4 gh4 = *reinterpret_cast<const f32x4*>(sF + 384 + drow), gl4 = *reinterpret_cast<const f32x4*>(sF + 448 + drow);

    f32x4 e4, d4;   // e^G, e^(G_last - G)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        e4[r] = __builtin_amdgcn_exp2f(gh4[r] + gl4[r]);
        d4[r] = __builtin_amdgcn_exp2f((sF[384 + 63] - gh4[r]) + (sF[448 + 63] - gl4[r]));
    }

    // B1, B2, the row and column sums of Z = B1 (q.k) + B2 (k.k), and the M part of dbeta
    f32x4 zrow = fz, mrow = fz;
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        float zc = 0.f;
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
                mma_planes<KP, KP, WP>(a, j, kk);
                mma_planes<KP, KP, WP>(q, j, qk);
            }
#pragma unroll
            for (int kb = 0; kb < PB; ++kb) {
                RawRow8<float> u;
                u.load(Ub + (16 * ct + l) * P + 32 * kb + 8 * g, true);
                bf16x8 j[WP];
                u.planes(j);
                mma_planes<KP, WP, WP>(o8[kb], j, dA);
                mma_planes<WP, WP, WP>(r8[kb], j, dM);
            }
            const int j = 16 * ct + l;
            const float gh = sF[384 + j], gl = sF[448 + j], rkj = sF[320 + j];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool diag = ct == w;
                const int i = 4 * g + r;
                float D = __builtin_amdgcn_exp2f((gh4[r] - gh) + (gl4[r] - gl));
                if (diag && l > i) D = 0.f;
                const float dm = (diag && l >= i) ? 0.f : -D * dM[r];
                const float b1 = p.scale * D * dA[r], kn = rk4[r] * rkj * kk[r], b2 = beta4[r] * dm;
                const float z = b1 * (rq4[r] * rkj * qk[r]) + b2 * kn;
                zrow[r] += z;
                mrow[r] += dm * kn;
                zc += z;
                sB1[(16 * w + i) * LB + j] = b1;
                sB2[(16 * w + i) * LB + j] = b2;
            }
        }
        zc = groups_sum(zc);
        if (g == 0) sCol[w * 64 + 16 * ct + l] = zc;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        zrow[r] = lanes_sum(zrow[r]);
        mrow[r] = lanes_sum(mrow[r]);
    }
    __syncthreads();

    // first operands from B1 (rows: dq; columns: dk) and B2 + B2^T (dk), with
    // the unit factors of the second operands' rows
    bf16x8 b1[2][WP], b1t[2][WP], b2[2][WP];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        float x[8], y[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = 32 * kb + 8 * g + e;
            const float rkj = sF[320 + j], rqj = sRq[j];
            x[e] = j <= irow ? sB1[irow * LB + j] * rkj : 0.f;
            y[e] = j >= irow ? sB1[j * LB + irow] * rqj : 0.f;
            z[e] = (j < irow ? sB2[irow * LB + j] : j > irow ? sB2[j * LB + irow] : 0.f) * rkj;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            bf16x2 t[WP];
            to_planes2<WP>(x[e], x[e + 1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b1[kb][i][e] = t[i][0]; b1[kb][i][e + 1] = t[i][1]; }
            to_planes2<WP>(y[e], y[e + 1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b1t[kb][i][e] = t[i][0]; b1t[kb][i][e + 1] = t[i][1]; }
            to_planes2<WP>(z[e], z[e + 1], t);
#pragma unroll
            for (int i = 0; i < WP; ++i) { b2[kb][i][e] = t[i][0]; b2[kb][i][e + 1] = t[i][1]; }
        }
    }

    // column tiles of dq and dk
    f32x4 accq[NT], acck[NT], qs = fz, ks = fz, us = fz, qd = fz, kd = fz;
    float tot = 0.f;
    const float* Sb = bp.S + ci * N * (int64_t)P;
    const float* Db = bp.dS + ci * N * (int64_t)P;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        f32x4 w1 = fz, w2 = fz, w3 = fz;
#pragma unroll
        for (int kb = 0; kb < PB; ++kb) {
            RawRow8<float> s, d;
            s.load(Sb + (16 * nt + l) * P + 32 * kb + 8 * g, true);
            d.load(Db + (16 * nt + l) * P + 32 * kb + 8 * g, true);
            bf16x8 s8[WP], d8[WP];
            s.planes(s8);
            d.planes(d8);
            mma_planes<KP, WP, WP>(o8[kb], s8, w1);
            mma_planes<WP, WP, WP>(r8[kb], s8, w2);
            mma_planes<WP, WP, WP>(u8[kb], d8, w3);
            if ((nt & 3) == w)
#pragma unroll
                for (int e = 0; e < 8; ++e) tot += s.get(e) * d.get(e);
        }
        // this tile's values of q and k at the result's places (unit rows)
        f32x4 qv = fz, kv = fz;
#pragma unroll
        for (int e = KP - 1; e >= 0; --e) {
            const int at = (e * 64 + 16 * w + 4 * g + (l >> 2)) * LK + 16 * nt + 4 * (l & 3);
            const bf16x4 x = lds_read_tr4(sQ + at), y = lds_read_tr4(sK + at);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                qv[r] += (float)x[r];
                kv[r] += (float)y[r];
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            qv[r] *= rq4[r];
            kv[r] *= rk4[r];
            w1[r] *= p.scale * e4[r];
            w2[r] *= e4[r];
            w3[r] *= d4[r];
            qs[r] += qv[r] * w1[r];
            ks[r] += kv[r] * w2[r];
            us[r] += kv[r] * w3[r];
            accq[nt][r] = w1[r];
            acck[nt][r] = w3[r] - beta4[r] * w2[r];
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            bf16x8 kt[KP], qt[KP];
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                const int at = (e * 64 + 32 * kb + 8 * g + (l >> 2)) * LK + 16 * nt + 4 * (l & 3);
                kt[e] = join8(lds_read_tr4(sK + at), lds_read_tr4(sK + at + 4 * LK));
                qt[e] = join8(lds_read_tr4(sQ + at), lds_read_tr4(sQ + at + 4 * LK));
            }
            mma_planes<WP, KP, WP>(b1[kb], kt, accq[nt]);
            mma_planes<WP, KP, WP>(b1t[kb], qt, acck[nt]);
            mma_planes<WP, KP, WP>(b2[kb], kt, acck[nt]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            qd[r] += qv[r] * accq[nt][r];
            kd[r] += kv[r] * acck[nt][r];
        }
    }
    // row sums over the tokens' columns
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        qs[r] = lanes_sum(qs[r]);
        ks[r] = lanes_sum(ks[r]);
        us[r] = lanes_sum(us[r]);
        qd[r] = lanes_sum(qd[r]);
        kd[r] = lanes_sum(kd[r]);
    }
    tot = groups_sum(lanes_sum(tot));
    if (lane == 0) sTot[w] = tot;

    // dq, dk through the unit rows: r (d - x (x.d))
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = drow + r;
            if (t >= nv) continue;
            float dq = accq[nt][r], dk = acck[nt][r];
            if (p.l2norm) {
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int e = KP - 1; e >= 0; --e) {
                    x += (float)sQ[(e * 64 + t) * LK + 16 * nt + l];
                    y += (float)sK[(e * 64 + t) * LK + 16 * nt + l];
                }
                dq = rq4[r] * (dq - x * rq4[r] * qd[r]);
                dk = rk4[r] * (dk - y * rk4[r] * kd[r]);
            }
            const int64_t at = ((t0 + t) * p.H + h) * N + 16 * nt + l;
            bp.dqe[at] = dq;
            bp.dke[at] = dk;
        }
    }
    // dbeta and dG of this wave's tokens
    if (l == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = drow + r;
            sG[t] = qs[r] - beta4[r] * ks[r] + zrow[r] - us[r];
            sUs[t] = us[r];
            if (t < nv) bp.dbeta[(t0 + t) * p.H + h] = sDb[t] - ks[r] + mrow[r];
        }
    }
    __syncthreads();
    if (w == 0) {
        double x = (double)sG[lane] - ((double)sCol[lane] + sCol[64 + lane] + sCol[128 + lane] + sCol[192 + lane]);
        const double u = wave_inclusive_sum_d((double)sUs[lane]);
        if (lane == 63) x += u + (double)sF[256] * ((double)sTot[0] + sTot[1] + sTot[2] + sTot[3]);
        const double s = wave_inclusive_sum_d(x);
        const double all = __shfl(s, 63);
        if (lane < nv) bp.dg[(t0 + lane) * p.H + h] = (float)(all - s + x);
    }
}

// dq and dk of a group of heads: the sum over its heads, in their order.
static __global__ __launch_bounds__(256) void delta_heads_kernel(const float* e, float* out, int64_t tokens, int H, int G, int N)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= tokens * G * N) return;
    const int64_t t = i / ((int64_t)G * N);
    const int j = (int)(i - t * G * N), gi = j / N, reach = H / G;
    const float* src = e + (t * H + (int64_t)gi * reach) * N + (j - gi * N);
    f32x4 s = *reinterpret_cast<const f32x4*>(src);
    for (int k = 1; k < reach; ++k) s += *reinterpret_cast<const f32x4*>(src + (int64_t)k * N);
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

template <typename IO, int N> struct GradLds {
    static constexpr size_t bytes = 2 * (size_t)DeltaPlanes<IO>::io * 64 * (N + 8) * 2 + (2 * 64 * 68 + 256 + 3 * 64 + 9 * 64 + 4) * 4;
};

template <typename IO, int N, int PB>
hipError_t launch_delta_grad(const DeltaBwdParams& bp, hipStream_t stream)
{
    auto* const kern = &delta_grad_kernel<IO, N, PB>;
    constexpr size_t lds = GradLds<IO, N>::bytes;
    static_assert(lds <= 160 * 1024, "a workgroup's LDS");
    static const hipError_t attr = delta_allow_lds(kern, lds);
    if (attr != hipSuccess) return attr;
    const int64_t blocks = (int64_t)bp.f.rows * bp.f.nc * bp.f.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), lds, stream, bp);
    return hipGetLastError();
}

template <typename IO, int N>
hipError_t bwd_n(const DeltaBwdParams& bp, hipStream_t stream)
{
    const DeltaParams& p = bp.f;
    hipError_t e = launch_delta_chunks<IO, N, true>(p, bp.ttf, bp.atf, stream);
    if (e != hipSuccess) return e;
    if ((e = launch_delta_walk<IO, N, 1, true>(p, bp.S, bp.U, stream)) != hipSuccess) return e;
    const int64_t blocks = (int64_t)p.rows * p.nc * p.H;
    if (blocks > 0) {
        hipLaunchKernelGGL((delta_pre_kernel<IO, N>), dim3((unsigned)blocks), dim3(256), 0, stream, bp);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.rows > 0) {
        auto* const back = &delta_back_kernel<IO, N>;
        constexpr size_t lds = WalkCfg<IO, N, 1>::total;
        static const hipError_t attr = delta_allow_lds(back, lds);
        if (attr != hipSuccess) return attr;
        const int64_t walks = ((int64_t)p.rows * p.H + 7) / 8 * 8 * (p.P / 16);
        hipLaunchKernelGGL(back, dim3((unsigned)walks), dim3(320), lds, stream, bp);
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
    if (p.cu != nullptr && p.L > 0) {
        const DeltaRest r = {{bp.dqe, bp.dke, bp.dv, bp.dg, bp.dbeta}, {p.H * p.N, p.H * p.N, p.H * p.P, p.H, p.H}};
        hipLaunchKernelGGL(delta_rest_kernel, dim3(p.rows + 1, 16), dim3(256), 0, stream, p, r);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.G != p.H && tokens > 0) {
        const int64_t n = (tokens * p.G * p.N / 4 + 255) / 256;
        hipLaunchKernelGGL(delta_heads_kernel, dim3((unsigned)n), dim3(256), 0, stream, bp.dqe, bp.dq, tokens, p.H, p.G, p.N);
        hipLaunchKernelGGL(delta_heads_kernel, dim3((unsigned)n), dim3(256), 0, stream, bp.dke, bp.dk, tokens, p.H, p.G, p.N);
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
