// Gated delta rule: the walk for calls with more (row, head, 16 columns) than
// the chip has CUs.
#pragma once

#include "m3_delta_walk.hpp"

namespace m3 {

// As delta_walk, for 16 NS columns to a workgroup, and with one state
// wavefront to 16 columns instead of four.  It runs the whole chain in its own
// registers: with the row order of tile_row a product's result is the next
// one's second operand as it lies, so neither LDS nor a barrier stands between
// the products.  A step takes it longer than four wavefronts together (four
// times their products), but it reads a quarter of what they read from LDS,
// which is what bounds a CU that runs several of them, and one K, T and set of
// factors serves NS of them.  The state waves leave S and U for
// four output waves, each with two row tiles of half the column groups (all
// groups of one tile read twice as much LDS, and buffers twice as large left no
// room for NS = 4 at N = 128, a third more there); Q S beside R and U,
// A U beside the state's product, two barriers a chunk.  bf16 calls only: K's
// planes of a float32 call would leave no room.
// 8 x 32 heads x 2048 tokens, P = 64: 228 us a call at N = 64 (delta_walk 334),
// of which 134 are this kernel's; 269 at N = 128 (369), of which 152: 660 MB at 4.3
// TB/s, 8850 cycles a chunk and CU, matrix cores busy for 39% of them, vector units
// 40%, LDS 35% and 10% in bank conflicts.  13 packed sequences of 20011 tokens, 32
// heads, N = P = 128: 345 to 370 us.
template <int N, int NS> struct WideCfg {
    static constexpr int WP = DeltaPlanes<bf16>::wide;
    static constexpr int KB = N / 32, NT = N / 16, waves = NS + 5;
    // S and U go to the output waves as planes, so that they need not split what
    // the state waves have split, or as float32, where planes would leave room for
    // one workgroup on a CU instead of two.  Calls over 2048 tokens, us, planes /
    // float32: NS = 4: 128 rows and heads at N = P = 128: 187 / 205, 256 at N =
    // 128, P = 64: 285 / 307; NS = 2: 96 at N = 64, P = 96: 180 / 157, 192: 290 /
    // 275.
    static constexpr bool PLANES = NS == 4;
    // bytes of one of two buffers, then per column group S and U
    static constexpr int k = 0, t = k + 64 * N * 2, f = t + kTriBlocks * WP * 1024, v = f + 5 * 256, buf = v + 64 * NS * 32;
    static constexpr int ex = 2 * buf, u = PLANES ? WP * KB * 1024 : KB * 2048, ex1 = u + (PLANES ? WP * 2048 : 4096), total = ex + NS * ex1;
};

template <int N, int NS>
__global__ __launch_bounds__(64 * (NS + 5)) void delta_wide_kernel(const DeltaParams p)
{
    using Cf = WideCfg<N, NS>;
    constexpr int WP = Cf::WP, KB = Cf::KB, NT = Cf::NT;
    extern __shared__ __attribute__((aligned(16))) char wlds[];

    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the workgroups of one (row, head) run on one XCD and share its L2
    const int nsl = p.P / (16 * NS);
    const int64_t idx = blockIdx.x >> 3;
    const int64_t unit = (idx / nsl) * 8 + (blockIdx.x & 7);
    if (unit >= (int64_t)p.rows * p.H) return;
    int b, h;
    delta_unit(p, unit, b, h);
    const int p0 = (int)(idx % nsl) * (16 * NS);
    const DeltaRow row = delta_row(p, b);
    const int64_t rec = delta_record(p, b, tid, 64 * Cf::waves, reinterpret_cast<int*>(wlds));
    const int nch = (int)((row.len + kDC - 1) / kDC);
    const int rs = p.G * N, vs = p.H * p.P;
    const int64_t ci0 = row.slot0 * p.H + h;
    const int nlast = (int)(row.len - (int64_t)(nch - 1) * kDC);   // tokens of the last chunk
    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};

    // what this wavefront has written to LDS is there, and s_barrier alone: the
    // release of __syncthreads would also wait for the loader's loads
    auto bar = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    if (wave == NS + 4) {   // loader: chunk c + 1 beside chunk c
        const bf16* kp = reinterpret_cast<const bf16*>(p.k) + (row.start * p.G + h / (p.H / p.G)) * N;
        const bf16* vp = reinterpret_cast<const bf16*>(p.v) + (row.start * p.H + h) * p.P + p0;
        auto stage = [&](int c) {
            char* buf = wlds + (c & 1) * Cf::buf;
            const int end = c == nch - 1 ? nlast - 1 : kDC - 1;   // last row to read
            const bf16 *kc = kp + (int64_t)c * kDC * rs, *vc = vp + (int64_t)c * kDC * vs;
            const float* fsrc = p.sc + (ci0 + (int64_t)c * p.H) * (kDScal * 64);
            to_lds16(buf + Cf::f, fsrc + 4 * lane);
            to_lds4(buf + Cf::f + 1024, fsrc + 256 + lane);
            constexpr int RPL = 512 / N, VPL = 32 / NS;   // K, V rows of one load
#pragma unroll
            for (int i = 0; i < 64 / RPL; ++i) {
                const int t = RPL * i + lane / (N / 8), j = k_block<N>(t, lane % (N / 8));
                to_lds16(buf + Cf::k + 1024 * i, kc + (t < end ? t : end) * rs + 8 * j);
            }
#pragma unroll
            for (int i = 0; i < 2 * NS; ++i) {
                const int t = VPL * i + lane / (2 * NS);
                to_lds16(buf + Cf::v + 1024 * i, vc + (t < end ? t : end) * vs + 8 * (lane % (2 * NS)));
            }
            const char* tsrc = reinterpret_cast<const char*>(p.tf + (ci0 + (int64_t)c * p.H) * (kTriBlocks * WP * 512));
#pragma unroll
            for (int i = 0; i < kTriBlocks * WP; ++i) to_lds16(buf + Cf::t + 1024 * i, tsrc + 1024 * i + 16 * lane);
        };
        if (nch > 0) stage(0);
        __builtin_amdgcn_s_waitcnt(0);
        bar();
        for (int c = 0; c < nch; ++c) {
            if (c + 1 < nch) stage(c + 1);
            bar();   // U
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0);
            bar();   // S
        }
        return;
    }

    if (wave >= NS) {   // output, as O^T: two row tiles of half the column groups
        const int w = wave - NS;
        const int tile[2] = {w & 1, 3 - (w & 1)};   // A spans one 32-token block there, and two
        constexpr int NG = NS / 2;
        const int cg0 = (w >> 1) * NG;
        const int t[2] = {tile_row(tile[0], l), tile_row(tile[1], l)};   // this lane's tokens
        const bf16* qp = reinterpret_cast<const bf16*>(p.q) + (row.start * p.G + h / (p.H / p.G)) * N + 8 * g;
        bf16* op = reinterpret_cast<bf16*>(p.o) + (row.start * p.H + h) * p.P + p0 + 16 * cg0 + 4 * g;
        bf16x8 q[2][KB][1];
        f32x4 a[3][2];   // [block][half]
        float fo[2];
        // (No load depends on a branch: where one might, a wait for the chunk's
        // operands would also wait for those of the chunk after it.)
        auto load_q = [&](int c) {
            c = c < nch ? c : nch - 1;
            const int end = c == nch - 1 ? nlast - 1 : kDC - 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16* qc = qp + (int64_t)c * kDC * rs + (t[i] < end ? t[i] : end) * rs;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) q[i][kb][0] = *reinterpret_cast<const bf16x8*>(qc + 32 * kb);
                fo[i] = p.sc[(ci0 + (int64_t)c * p.H) * (kDScal * 64) + 192 + t[i]];
            }
        };
        auto load_a = [&](int c) {
            c = c < nch ? c : nch - 1;
            const float* src = p.af + (ci0 + (int64_t)c * p.H) * (int64_t)kTriValues + 4 * lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                a[0][j] = *reinterpret_cast<const f32x4*>(src + low_block(tile[0], 0) * 512 + 256 * j);
                a[1][j] = *reinterpret_cast<const f32x4*>(src + low_block(tile[1], 0) * 512 + 256 * j);
                a[2][j] = *reinterpret_cast<const f32x4*>(src + low_block(tile[1], 1) * 512 + 256 * j);
            }
        };
        // block kb of the `blocks` of S or U at s
        auto get = [&](const char* s, int kb, int blocks, bf16x8 (&x)[WP]) {
            if constexpr (Cf::PLANES) {
#pragma unroll
                for (int j = 0; j < WP; ++j) x[j] = *reinterpret_cast<const bf16x8*>(s + (j * blocks + kb) * 1024);
            } else {
                cut8(*reinterpret_cast<const f32x4*>(s + kb * 2048), *reinterpret_cast<const f32x4*>(s + kb * 2048 + 1024), x);
            }
        };
        if (nch > 0) {
            load_q(0);
            load_a(0);
        }
        bar();
        const char* ex = wlds + Cf::ex + cg0 * Cf::ex1 + 16 * lane;
        for (int c = 0; c < nch; ++c) {
            f32x4 acc[2][NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                acc[0][i] = fz;
                acc[1][i] = fz;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 s8[1][WP];
                    get(ex + i * Cf::ex1, kb, KB, s8[0]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma_tiles<1, WP, 1, WP>(s8, q[k][kb], &acc[k][i]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[k][i][r] *= fo[k];
            }
            load_q(c + 1);
            bf16x8 a8[3][WP];
#pragma unroll
            for (int i = 0; i < 3; ++i) cut8(a[i][0], a[i][1], a8[i]);
            bar();   // U
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    bf16x8 u8[1][WP];
                    get(ex + i * Cf::ex1 + Cf::u, kb, 2, u8[0]);
                    if (kb == 0) mma_tiles<1, WP, WP, WP>(u8, a8[0], &acc[0][i]);
                    mma_tiles<1, WP, WP, WP>(u8, a8[1 + kb], &acc[1][i]);
                }
            load_a(c + 1);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (t[k] < (c == nch - 1 ? nlast : kDC)) {
                    bf16* oc = op + ((int64_t)c * kDC + t[k]) * vs;
#pragma unroll
                    for (int i = 0; i < NG; ++i) gstore4(oc + 16 * i, acc[k][i]);
                }
            bar();   // S
        }
        return;
    }

    const int cg = wave;   // column group
    char* ex = wlds + Cf::ex + cg * Cf::ex1 + 16 * lane;

    // state: tile i holds rows tile_row(i, 4 g + r) of the state, column l
    const int col = p0 + 16 * cg + l;
    f32x4 S[NT];
    const float* hin = p.h_in != nullptr && rec >= 0 ? p.h_in + ((rec * p.H + h) * N + 8 * g) * p.P + col : nullptr;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            S[i][r] = hin != nullptr ? hin[(32 * (i >> 1) + 4 * (i & 1) + r) * p.P] : 0.f;
            if (rec == -2) S[i][r] = __builtin_nanf("");   // the record belongs to an earlier row
        }
    bf16x8 s8[KB][WP];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) planes8<WP>(S[2 * kb], S[2 * kb + 1], s8[kb]);
    auto put_state = [&]() {
        if constexpr (Cf::PLANES) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x8*>(ex + (j * KB + kb) * 1024) = s8[kb][j];
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(ex + i * 1024) = S[i];
        }
    };
    put_state();
    bar();

    for (int c = 0; c < nch; ++c) {
        const char* buf = wlds + (c & 1) * Cf::buf;
        // R = beta V - sp (K S)
        f32x4 P[4] = {fz, fz, fz, fz};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 k8[4][1];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const int t = tile_row(rt, l);
                k8[rt][0] = *reinterpret_cast<const bf16x8*>(buf + Cf::k + t * (2 * N) + 16 * k_block<N>(t, 4 * kb + g));
            }
            mma_tiles<4, 1, WP, WP>(k8, s8[kb], P);
        }
        bf16x8 r8[2][WP];
        const float* f = reinterpret_cast<const float*>(buf + Cf::f) + 8 * g;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const int t0 = 32 * (rt >> 1) + 4 * (rt & 1);
            const f32x4 fb = *reinterpret_cast<const f32x4*>(f + t0), fp = *reinterpret_cast<const f32x4*>(f + 64 + t0);
            const bf16x4 v = lds_read_tr4(reinterpret_cast<const bf16*>(buf + Cf::v) + (t0 + 8 * g + (l >> 2)) * (16 * NS) +
                                          16 * cg + 4 * (l & 3));
#pragma unroll
            for (int r = 0; r < 4; ++r) P[rt][r] = fb[r] * (float)v[r] - fp[r] * P[rt][r];
        }
        planes8<WP>(P[0], P[1], r8[0]);
        planes8<WP>(P[2], P[3], r8[1]);
        // U = T R
        f32x4 U[4] = {fz, fz, fz, fz};
        {
            const char* tb = buf + Cf::t + 16 * lane;
            bf16x8 t4[4][WP], t2[2][WP];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < WP; ++j) t4[i][j] = *reinterpret_cast<const bf16x8*>(tb + (i * WP + j) * 1024);
            mma_tiles<4, WP, WP, WP>(t4, r8[0], U);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < WP; ++j) t2[i][j] = *reinterpret_cast<const bf16x8*>(tb + ((4 + i) * WP + j) * 1024);
            mma_tiles<2, WP, WP, WP>(t2, r8[1], U + 2);
        }
        if constexpr (Cf::PLANES) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                bf16x8 o[WP];
                planes8<WP>(U[2 * kb], U[2 * kb + 1], o);
#pragma unroll
                for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x8*>(ex + Cf::u + (2 * j + kb) * 1024) = o[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(ex + Cf::u + i * 1024) = U[i];
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 fu = *reinterpret_cast<const f32x4*>(f + 128 + 32 * (rt >> 1) + 4 * (rt & 1));
#pragma unroll
            for (int r = 0; r < 4; ++r) U[rt][r] *= fu[r];
        }
        planes8<WP>(U[0], U[1], r8[0]);
        planes8<WP>(U[2], U[3], r8[1]);
        bar();   // U
        // S <- e^G_last S + K^T (d U)
        const float eL = *reinterpret_cast<const float*>(buf + Cf::f + 1024 + 4 * lane);
        constexpr int TN = NT < 4 ? NT : 4;   // tiles in turn
#pragma unroll
        for (int i0 = 0; i0 < NT; i0 += TN) {
            f32x4 acc[TN];
#pragma unroll
            for (int i = 0; i < TN; ++i) acc[i] = fz;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                bf16x8 kt[TN][1];
                const int t = 32 * kb + 8 * g + (l >> 2);
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    const int j4 = 4 * ((i0 + i) >> 1) + (l & 3);
                    const char* src = buf + Cf::k + 8 * (i & 1);
                    kt[i][0] = join8(lds_read_tr4(reinterpret_cast<const bf16*>(src + t * (2 * N) + 16 * k_block<N>(t, j4))),
                                     lds_read_tr4(reinterpret_cast<const bf16*>(src + (t + 4) * (2 * N) + 16 * k_block<N>(t + 4, j4))));
                }
                mma_tiles<TN, 1, WP, WP>(kt, r8[kb], acc);
            }
#pragma unroll
            for (int i = 0; i < TN; i += 2) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    S[i0 + i][r] = eL * S[i0 + i][r] + acc[i][r];
                    S[i0 + i + 1][r] = eL * S[i0 + i + 1][r] + acc[i + 1][r];
                }
                planes8<WP>(S[i0 + i], S[i0 + i + 1], s8[(i0 + i) / 2]);
            }
        }
        put_state();
        bar();   // S
    }
    if (p.h_out != nullptr && rec >= 0) {
        float* ho = p.h_out + ((rec * p.H + h) * N + 8 * g) * p.P + col;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) ho[(32 * (i >> 1) + 4 * (i & 1) + r) * p.P] = S[i][r];
    }
}

template <int N, int NS>
hipError_t launch_delta_wide(const DeltaParams& p, hipStream_t stream)
{
    using Cf = WideCfg<N, NS>;
    auto* const kern = &delta_wide_kernel<N, NS>;
    static_assert(Cf::total <= 160 * 1024, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    const hipError_t attr = delta_allow_lds(kern, Cf::total, done);
    if (attr != hipSuccess) return attr;
    const int64_t blocks = ((int64_t)p.rows * p.H + 7) / 8 * 8 * (p.P / (16 * NS));
    const size_t lds = Cf::total;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * Cf::waves), lds, stream, p);
    return hipGetLastError();
}

}  // namespace m3
