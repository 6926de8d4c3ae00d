// Gated delta rule: the kernel that makes what a chunk's products need and
// no state enters (T, A, per-token factors), and the walk over the chunks.
#pragma once

#include "m3_delta.hpp"

namespace m3 {

// acc += A B for 16 x 16 float32 tiles in LDS (row-major, leading dimensions
// lda, ldb): lane (l, g) supplies A[l][k], B[k][l] of k = 4 kk + g.
__device__ __forceinline__ void tile_mm(const float* A, int lda, const float* B, int ldb, int l, int g, f32x4& acc)
{
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(A[l * lda + 4 * kk + g], B[(4 * kk + g) * ldb + l], acc, 0, 0, 0);
}
__device__ __forceinline__ void tile_put(float* C, int ldc, int l, int g, const f32x4& v)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) C[(4 * g + r) * ldc + l] = v[r];
}

// What one chunk of one head needs besides its rows:
//   T = (I + M)^-1, A = scale D o Q K^T (rows divided by their norms where the
//   call asks for it), and per token  beta | beta e^G / |k| | e^(G_last - G) /
//   |k| | scale e^G / |q|, then e^G_last.
// One workgroup of four waves per chunk and head, wave w on rows 16w..16w+15.
// K and Q rows are the operands as they lie in memory (lane: one row, 8
// columns), so the two 64 x 64 products take no LDS.  M is inverted by blocks:
// substitution inside the four 16 x 16 diagonal blocks (one column per lane,
// in registers), then pairs of blocks joined, [[A,0],[C,B]]^-1 = [[A^-1,0],
// [-B^-1 C A^-1, B^-1]], with float32 matrix instructions.  Substitution and
// not the product (I-M)(I+M^2)(I+M^4).., whose terms cancel where keys repeat.
// G is summed in 64 bits and kept as two float32 in units of log 2: the
// difference of two sums keeps float32's relative precision after a token
// whose decay is near zero.
template <typename IO, int N, bool BWD>
__global__ __launch_bounds__(256) void delta_chunk_kernel(const DeltaParams p, bf16* ttf, bf16* atf)
{
    constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide, OP = DeltaPlanes<IO>::out;
    constexpr int AP = BWD ? WP : OP;     // the gradient's path is float32 throughout
    constexpr int KB = N / 32, LD = 68;
    __shared__ float sGh[64], sGl[64], sBeta[64], sRk[64], sRq[64], sE[64], sD[64];
    __shared__ __attribute__((aligned(16))) float sM[64 * LD];
    __shared__ __attribute__((aligned(16))) float sT[64 * LD];   // A first, then T
    __shared__ float sX[32 * 36];

    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bid = blockIdx.x;
    const int h = (int)(bid % p.H);
    const int64_t bc = bid / p.H;
    const int c = (int)(bc % p.nc), b = (int)(bc / p.nc);
    const DeltaRow row = delta_row(p, b);
    if ((int64_t)c * kDC >= row.len) return;
    const int64_t t0 = row.start + (int64_t)c * kDC;
    const int nv = row.len - (int64_t)c * kDC < kDC ? (int)(row.len - (int64_t)c * kDC) : kDC;
    const int64_t ci = (row.slot0 + c) * p.H + h;
    const int hg = h / (p.H / p.G);
    const IO* kb_ = reinterpret_cast<const IO*>(p.k) + (t0 * p.G + hg) * N;
    const IO* qb_ = reinterpret_cast<const IO*>(p.q) + (t0 * p.G + hg) * N;
    const int64_t rs = (int64_t)p.G * N;   // row stride of q and k

    // this wave's rows of K and Q
    RawRow8<IO> kr[KB], qr[KB];
    const int irow = 16 * w + l;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        kr[kb].load(kb_ + irow * rs + 32 * kb + 8 * g, irow < nv);
        qr[kb].load(qb_ + irow * rs + 32 * kb + 8 * g, irow < nv);
    }

    if (w == 0) {
        const bool ok = lane < nv;
        float gv = ok ? p.g[(t0 + lane) * p.H + h] : 0.f;
        const float bv = ok ? p.beta[(t0 + lane) * p.H + h] : 0.f;
        gv = gv < -1024.f ? -1024.f : gv;   // exp is zero there; keeps -inf out of differences
        double s = (double)gv * 1.4426950408889634;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double t = __shfl_up(s, o);
            if (lane >= o) s += t;
        }
        const double last = __shfl(s, 63);
        sGh[lane] = (float)s;
        sGl[lane] = (float)(s - (double)(float)s);
        sBeta[lane] = bv;
        sE[lane] = exp2f((float)s);
        sD[lane] = exp2f((float)(last - s));
        if (!p.l2norm) {
            sRk[lane] = 1.f;
            sRq[lane] = 1.f;
        }
    }

    // K K^T and Q K^T, column tiles 0..w
    f32x4 kk[4], qk[4];
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};
    for (int ct = 0; ct < 4; ++ct) {
        kk[ct] = fz;
        qk[ct] = fz;
    }
    float q2 = 0.f;
    if (p.l2norm) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 8; ++e) q2 += qr[kb].get(e) * qr[kb].get(e);
        q2 += __shfl_xor(q2, 16);
        q2 += __shfl_xor(q2, 32);
        if (g == 0) sRq[irow] = irow < nv ? 1.f / sqrtf(q2 + p.eps) : 0.f;
    }
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        if (ct > w) continue;   // wave-uniform
        const int jrow = 16 * ct + l;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            RawRow8<IO> jr;
            jr.load(kb_ + jrow * rs + 32 * kb + 8 * g, jrow < nv);
            bf16x8 a[KP], qa[KP], j[KP];
            kr[kb].planes(a);
            qr[kb].planes(qa);
            jr.planes(j);
            mma_planes<KP, KP, WP>(a, j, kk[ct]);
            mma_planes<KP, KP, WP>(qa, j, qk[ct]);
        }
    }
    if (p.l2norm) {
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            if (ct != w) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (l == 4 * g + r) {   // the diagonal: |k|^2
                    const int i = 16 * w + l;
                    sRk[i] = i < nv ? 1.f / sqrtf(kk[ct][r] + p.eps) : 0.f;
                }
        }
    }
    __syncthreads();

    // M and A; entries above the diagonal stay out
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
        if (ct > w) continue;
        const int j = 16 * ct + l;
        const float gh = sGh[j], gl = sGl[j], rkj = sRk[j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * w + 4 * g + r;
            const float D = exp2f((sGh[i] - gh) + (sGl[i] - gl)) * rkj;
            sM[i * LD + j] = j < i ? sBeta[i] * sRk[i] * D * kk[ct][r] : 0.f;
            sT[i * LD + j] = j <= i ? p.scale * sRq[i] * D * qk[ct][r] : 0.f;
        }
    }
    if (w == 0) {   // per-token factors
        float* sc = p.sc + ci * (kDScal * 64);
        const float rk = sRk[lane], e = sE[lane], bv = sBeta[lane];
        sc[lane] = bv;
        sc[64 + lane] = bv * e * rk;
        sc[128 + lane] = sD[lane] * rk;
        sc[192 + lane] = p.scale * e * sRq[lane];
        if (lane == 0) sc[256] = sE[63];
        if (BWD) sc[320 + lane] = rk;
    }
    __syncthreads();

    // A in operand order: the wave's own rows
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        if (kb > (w >> 1)) continue;
        bf16x8 o[AP];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = 32 * kb + 8 * g + e;
            bf16 t[AP];
            to_planes<AP>(col <= irow ? sT[irow * LD + col] : 0.f, t);
#pragma unroll
            for (int i = 0; i < AP; ++i) o[i][e] = t[i];
        }
        if (!BWD)
#pragma unroll
            for (int i = 0; i < AP; ++i)
                *reinterpret_cast<bf16x8*>(p.af + ci * (kTriBlocks * AP * 512) + ((low_block(w, kb) * AP + i) * 64 + lane) * 8) = o[i];
    }
    if (BWD) {   // A^T: row j of the transpose is column j
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb < (w >> 1)) continue;
            bf16x8 o[AP];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int col = 32 * kb + 8 * g + e;
                bf16 t[AP];
                to_planes<AP>(col >= irow ? sT[col * LD + irow] : 0.f, t);
#pragma unroll
                for (int i = 0; i < AP; ++i) o[i][e] = t[i];
            }
#pragma unroll
            for (int i = 0; i < AP; ++i)
                *reinterpret_cast<bf16x8*>(atf + ci * (kTriBlocks * AP * 512) + ((up_block(w, kb) * AP + i) * 64 + lane) * 8) = o[i];
        }
    }
    __syncthreads();   // sT is T from here

    // diagonal block of rows 16w: column l of its inverse
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == l ? 1.f : 0.f;
#pragma unroll
            for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
                const f32x4 m = *reinterpret_cast<const f32x4*>(&sM[(16 * w + i) * LD + 16 * w + 4 * j4]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * j4 + e < i) s -= m[e] * x[4 * j4 + e];
            }
            x[i] = s;
        }
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sT[(16 * w + i) * LD + 16 * w + l] = x[i];
        }
    }
    __syncthreads();
    // blocks (1,0) and (3,2)
    if (w < 2) {
        f32x4 x = fz;
        tile_mm(&sM[(32 * w + 16) * LD + 32 * w], LD, &sT[32 * w * LD + 32 * w], LD, l, g, x);
        tile_put(sX + w * 320, 20, l, g, x);
    }
    __syncthreads();
    if (w < 2) {
        f32x4 x = fz;
        tile_mm(&sT[(32 * w + 16) * LD + 32 * w + 16], LD, sX + w * 320, 20, l, g, x);
        tile_put(&sT[(32 * w + 16) * LD + 32 * w], LD, l, g, -x);
    }
    __syncthreads();
    // the 32 x 32 block below: X = C A^-1, then -B^-1 X
    {
        const int ta = w >> 1, tb = w & 1;
        f32x4 x = fz;
        for (int k = tb; k < 2; ++k)
            tile_mm(&sM[(32 + 16 * ta) * LD + 16 * k], LD, &sT[16 * k * LD + 16 * tb], LD, l, g, x);
        tile_put(sX + 16 * ta * 36 + 16 * tb, 36, l, g, x);
        __syncthreads();
        x = fz;
        for (int k = 0; k <= ta; ++k)
            tile_mm(&sT[(32 + 16 * ta) * LD + 32 + 16 * k], LD, sX + 16 * k * 36 + 16 * tb, 36, l, g, x);
        tile_put(&sT[(32 + 16 * ta) * LD + 16 * tb], LD, l, g, -x);
    }
    __syncthreads();

    // T in operand order
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        if (kb > (w >> 1)) continue;
        bf16x8 o[WP];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = 32 * kb + 8 * g + e;
            bf16 t[WP];
            to_planes<WP>(col <= irow ? sT[irow * LD + col] : 0.f, t);
#pragma unroll
            for (int i = 0; i < WP; ++i) o[i][e] = t[i];
        }
#pragma unroll
        for (int i = 0; i < WP; ++i)
            *reinterpret_cast<bf16x8*>(p.tf + ci * (kTriBlocks * WP * 512) + ((low_block(w, kb) * WP + i) * 64 + lane) * 8) = o[i];
    }
    if (BWD) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb < (w >> 1)) continue;
            bf16x8 o[WP];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int col = 32 * kb + 8 * g + e;
                bf16 t[WP];
                to_planes<WP>(col >= irow ? sT[col * LD + irow] : 0.f, t);
#pragma unroll
                for (int i = 0; i < WP; ++i) o[i][e] = t[i];
            }
#pragma unroll
            for (int i = 0; i < WP; ++i)
                *reinterpret_cast<bf16x8*>(ttf + ci * (kTriBlocks * WP * 512) + ((up_block(w, kb) * WP + i) * 64 + lane) * 8) = o[i];
        }
    }
}

// LDS of the walk, in bf16 elements.
template <typename IO, int N, int NCG> struct WalkLds {
    static constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide, OP = DeltaPlanes<IO>::out;
    static constexpr int LK = N + 8, LT = 72, C = 16 * NCG;
    static constexpr int k = 0, s = k + KP * 64 * LK, r = s + WP * C * LK, u2 = r + WP * C * LT, u = u2 + WP * C * LT,
                         total = u + OP * C * LT;
    static constexpr size_t bytes = 2 * (size_t)total;
};

// The walk over one row's chunks for one head and 16 NCG columns of V.
//
// Per chunk, wave w of a column group of 16 holds rows 16w..16w+15 of the
// chunk and rows n of the state in tiles w, w + 4:
//   P = K S, Q S        (operands: its K and Q rows from memory, S from LDS)
//   U = T (beta V - sp P)
//   S = e^G_last S + K^T (d U),  O = e Q S + A U
// three stages with a barrier after each, because the next stage's second
// operand is what all four waves have just made.  Everything that does not
// depend on the state (rows, T, A, factors) is read straight into operand
// registers one chunk ahead.  The walk's time is the latency of this chain,
// not its arithmetic, so a call with few (row, head) pairs takes 16 columns per
// workgroup and spreads over the chip.
// TRAIN: writes each chunk's first state and U for the gradient instead of O.
template <typename IO, int N, int NCG, bool TRAIN>
__global__ __launch_bounds__(256 * NCG) void delta_walk_kernel(const DeltaParams p, float* Sbuf, float* Ubuf)
{
    using Ld = WalkLds<IO, N, NCG>;
    constexpr int KP = Ld::KP, WP = Ld::WP, OP = Ld::OP, LK = Ld::LK, LT = Ld::LT, C = Ld::C;
    constexpr int KB = N / 32, NT = N / 16, TI = (NT + 3) / 4;
    extern __shared__ __attribute__((aligned(16))) bf16 dlds[];
    __shared__ int sflag;
    bf16 *sK = dlds + Ld::k, *sS = dlds + Ld::s, *sR = dlds + Ld::r, *sU2 = dlds + Ld::u2, *sU = dlds + Ld::u;

    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w = wave & 3, cg = wave >> 2;
    // the slices of one (row, head) run on one XCD and share its L2
    const int nsl = p.P / C;
    const int64_t idx = blockIdx.x >> 3;
    const int64_t unit = (idx / nsl) * 8 + (blockIdx.x & 7);
    if (unit >= (int64_t)p.rows * p.H) return;
    int64_t b64, h64;
    split_bh(unit, p.H, b64, h64);
    const int b = (int)b64, h = (int)h64;
    const int p0 = (int)(idx % nsl) * C + cg * 16;   // this wave's first column
    const DeltaRow row = delta_row(p, b);
    const int64_t rec = TRAIN ? b : delta_record(p, b, tid, 256 * NCG, &sflag);
    const int nch = (int)((row.len + kDC - 1) / kDC);
    const int hg = h / (p.H / p.G);
    const int64_t rs = (int64_t)p.G * N, vs = (int64_t)p.H * p.P;
    const IO* kp = reinterpret_cast<const IO*>(p.k) + (row.start * p.G + hg) * N;
    const IO* qp = reinterpret_cast<const IO*>(p.q) + (row.start * p.G + hg) * N;
    const IO* vp = reinterpret_cast<const IO*>(p.v) + (row.start * p.H + h) * p.P + p0 + l;
    IO* op = reinterpret_cast<IO*>(p.o) + (row.start * p.H + h) * p.P + p0 + l;

    // state tiles: rows 16 (w + 4 i) + 4 g + r, column l
    f32x4 S[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int n0 = 16 * (w + 4 * i) + 4 * g;
        const bool mine = w + 4 * i < NT;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            S[i][r] = mine && p.h_in != nullptr && rec >= 0
                          ? p.h_in[((rec * p.H + h) * N + n0 + r) * p.P + p0 + l] : 0.f;
            if (rec == -2) S[i][r] = __builtin_nanf("");   // the record belongs to an earlier row
        }
    }
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            if (w + 4 * i >= NT) continue;
            bf16x4 o[WP];
            to_planes4<WP>(S[i], o);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                *reinterpret_cast<bf16x4*>(sS + (j * C + cg * 16 + l) * LK + 16 * (w + 4 * i) + 4 * g) = o[j];
        }
    };
    put_state();

    const int irow = 16 * w + l;          // operand row of this lane
    const int drow = 16 * w + 4 * g;      // first result row of this lane
    RawRow8<IO> kr[KB], qr[KB];
    bf16x8 tf[2][WP], af[2][OP];
    float v[4];
    f32x4 fb, fp, fu, fo;
    float eL;
    const int nb = (w >> 1) + 1;          // 32-column blocks of this wave's rows in T and A
    auto load_k = [&](int c) {
        const int64_t t = (int64_t)c * kDC + irow;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) kr[kb].load(kp + t * rs + 32 * kb + 8 * g, t < row.len);
    };
    auto load_q = [&](int c) {
        const int64_t t = (int64_t)c * kDC + irow;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) qr[kb].load(qp + t * rs + 32 * kb + 8 * g, t < row.len);
    };
    auto load_v = [&](int c) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t t = (int64_t)c * kDC + drow + r;
            v[r] = t < row.len ? to_f32(vp[t * vs]) : 0.f;
        }
    };
    auto load_t = [&](int c) {
        const bf16* src = p.tf + ((row.slot0 + c) * p.H + h) * (kTriBlocks * WP * 512) + lane * 8;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb < nb)
#pragma unroll
                for (int i = 0; i < WP; ++i)
                    tf[kb][i] = *reinterpret_cast<const bf16x8*>(src + (low_block(w, kb) * WP + i) * 512);
    };
    auto load_a = [&](int c) {
        const bf16* src = p.af + ((row.slot0 + c) * p.H + h) * (kTriBlocks * OP * 512) + lane * 8;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb < nb)
#pragma unroll
                for (int i = 0; i < OP; ++i)
                    af[kb][i] = *reinterpret_cast<const bf16x8*>(src + (low_block(w, kb) * OP + i) * 512);
    };
    auto load_f = [&](int c) {
        const float* src = p.sc + ((row.slot0 + c) * p.H + h) * (kDScal * 64);
        fb = *reinterpret_cast<const f32x4*>(src + drow);
        fp = *reinterpret_cast<const f32x4*>(src + 64 + drow);
        fu = *reinterpret_cast<const f32x4*>(src + 128 + drow);
        fo = *reinterpret_cast<const f32x4*>(src + 192 + drow);
        eL = src[256];
    };
    if (nch > 0) {
        load_k(0);
        if (!TRAIN) load_q(0);
        load_v(0);
        load_f(0);
        load_t(0);
        if (!TRAIN) load_a(0);
    }
    __syncthreads();

    for (int c = 0; c < nch; ++c) {
        const int64_t ci = (row.slot0 + c) * p.H + h;
        if (TRAIN) {
#pragma unroll
            for (int i = 0; i < TI; ++i)
                if (w + 4 * i < NT)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        Sbuf[(ci * N + 16 * (w + 4 * i) + 4 * g + r) * p.P + p0 + l] = S[i][r];
        }
        // stage 1
        f32x4 aP = {0.f, 0.f, 0.f, 0.f}, aQ = aP;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 k8[KP], s8[WP];
            kr[kb].planes(k8);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                s8[j] = *reinterpret_cast<const bf16x8*>(sS + (j * C + cg * 16 + l) * LK + 32 * kb + 8 * g);
            mma_planes<KP, WP, WP>(k8, s8, aP);
            if (!TRAIN) {
                bf16x8 q8[KP];
                qr[kb].planes(q8);
                mma_planes<KP, WP, OP>(q8, s8, aQ);
            }
            if (cg == 0) {
#pragma unroll
                for (int j = 0; j < KP; ++j)
                    *reinterpret_cast<bf16x8*>(sK + (j * 64 + irow) * LK + 32 * kb + 8 * g) = k8[j];
            }
        }
        {
            f32x4 R;
#pragma unroll
            for (int r = 0; r < 4; ++r) R[r] = fb[r] * v[r] - fp[r] * aP[r];
            bf16x4 o[WP];
            to_planes4<WP>(R, o);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                *reinterpret_cast<bf16x4*>(sR + (j * C + cg * 16 + l) * LT + drow) = o[j];
        }
        const f32x4 cu_ = fu, co_ = fo;
        const float ceL = eL;
        if (c + 1 < nch) {
            load_k(c + 1);
            if (!TRAIN) load_q(c + 1);
            load_v(c + 1);
            load_f(c + 1);
        }
        __syncthreads();
        // stage 2
        f32x4 aU = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb < nb) {
                bf16x8 r8[WP];
#pragma unroll
                for (int j = 0; j < WP; ++j)
                    r8[j] = *reinterpret_cast<const bf16x8*>(sR + (j * C + cg * 16 + l) * LT + 32 * kb + 8 * g);
                mma_planes<WP, WP, WP>(tf[kb], r8, aU);
            }
        {
            f32x4 u2;
#pragma unroll
            for (int r = 0; r < 4; ++r) u2[r] = cu_[r] * aU[r];
            bf16x4 o[WP];
            to_planes4<WP>(u2, o);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                *reinterpret_cast<bf16x4*>(sU2 + (j * C + cg * 16 + l) * LT + drow) = o[j];
            if (!TRAIN) {
                bf16x4 q[OP];
                to_planes4<OP>(aU, q);
#pragma unroll
                for (int j = 0; j < OP; ++j)
                    *reinterpret_cast<bf16x4*>(sU + (j * C + cg * 16 + l) * LT + drow) = q[j];
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) Ubuf[(ci * 64 + drow + r) * p.P + p0 + l] = aU[r];
            }
        }
        if (c + 1 < nch) load_t(c + 1);
        __syncthreads();
        // stage 3
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            if (w + 4 * i >= NT) continue;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                bf16x8 u8[WP], kt[KP];
#pragma unroll
                for (int j = 0; j < WP; ++j)
                    u8[j] = *reinterpret_cast<const bf16x8*>(sU2 + (j * C + cg * 16 + l) * LT + 32 * kb + 8 * g);
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    const bf16* src = sK + (j * 64 + 32 * kb + 8 * g + (l >> 2)) * LK + 16 * (w + 4 * i) + 4 * (l & 3);
                    const bf16x4 lo = lds_read_tr4(src), hi = lds_read_tr4(src + 4 * LK);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { kt[j][e] = lo[e]; kt[j][4 + e] = hi[e]; }
                }
                mma_planes<KP, WP, WP>(kt, u8, acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = ceL * S[i][r] + acc[r];
        }
        put_state();
        if (!TRAIN) {
            f32x4 aO;
#pragma unroll
            for (int r = 0; r < 4; ++r) aO[r] = co_[r] * aQ[r];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb < nb) {
                    bf16x8 u8[OP];
#pragma unroll
                    for (int j = 0; j < OP; ++j)
                        u8[j] = *reinterpret_cast<const bf16x8*>(sU + (j * C + cg * 16 + l) * LT + 32 * kb + 8 * g);
                    mma_planes<OP, OP, OP>(af[kb], u8, aO);
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t t = (int64_t)c * kDC + drow + r;
                if (t < row.len) op[t * vs] = from_f32<IO>(aO[r]);
            }
            if (c + 1 < nch) load_a(c + 1);
        }
        __syncthreads();
    }

    if (!TRAIN && p.h_out != nullptr && rec >= 0) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    p.h_out[((rec * p.H + h) * N + 16 * (w + 4 * i) + 4 * g + r) * p.P + p0 + l] = S[i][r];
    }
}

template <typename F> hipError_t delta_allow_lds(F* kern, size_t bytes)
{
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes);
    (void)hipGetLastError();
    return e;
}

template <typename IO, int N, bool BWD>
hipError_t launch_delta_chunks(const DeltaParams& p, bf16* ttf, bf16* atf, hipStream_t stream)
{
    const int64_t blocks = (int64_t)p.rows * p.nc * p.H;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_chunk_kernel<IO, N, BWD>), dim3((unsigned)blocks), dim3(256), 0, stream, p, ttf, atf);
    return hipGetLastError();
}

template <typename IO, int N, int NCG, bool TRAIN>
hipError_t launch_delta_walk(const DeltaParams& p, float* Sbuf, float* Ubuf, hipStream_t stream)
{
    auto* const kern = &delta_walk_kernel<IO, N, NCG, TRAIN>;
    constexpr size_t lds = WalkLds<IO, N, NCG>::bytes;
    static const hipError_t attr = delta_allow_lds(kern, lds);
    if (attr != hipSuccess) return attr;
    const int64_t units = ((int64_t)p.rows * p.H + 7) / 8 * 8;
    const int64_t blocks = units * (p.P / (16 * NCG));
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256 * NCG), lds, stream, p, Sbuf, Ubuf);
    return hipGetLastError();
}

}  // namespace m3
