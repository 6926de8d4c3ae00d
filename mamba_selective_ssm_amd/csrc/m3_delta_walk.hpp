// Gated delta rule: the walk over a row's chunks.
#pragma once

#include <atomic>
#include <type_traits>

#include "m3_delta.hpp"

namespace m3 {

// The walk over one row's chunks for one head and 16 columns of V.
//
// Per chunk:  R = beta V - sp (K S) | U = T R | S <- e^G_last S + K^T (d U),
// and O = so (Q S) + A U with the chunk's first S.  Each product needs the one
// before it, so the walk's time is this chain's, chunk after chunk, and all
// that is not on it is kept out of it:
//   - four state wavefronts run the chain, wave w on row tile w
//     of each product; a result leaves as planes in operand order (tile_row),
//     so that all four read it back with plain 16-byte reads after a barrier;
//   - a loader wavefront moves K, T, V and the factors from memory straight to
//     LDS, NBUF - 1 chunks ahead (float32 K through its registers, where it is
//     split into planes: read two chunks ahead, 29 us for 37 at 32 slices of 13
//     chunks, N = 64);
//   - three output wavefronts make O from the planes of S and from U, Q S
//     while the state goes through T, A U during the next chunk's first stage:
//     row tiles 0 and 1, tile 2, and tile 3, which A spans with two blocks each.
//     A and U come as float32 and are split into planes here, half of A beside
//     each of the later stages, where these wavefronts have the least to do (all
//     of A beside one of them: 2 us more at 256 slices of N = 64, below, or 10
//     to 40 us at 128 slices of 1024 chunks, N = 128).  With two wavefronts, row
//     tiles 0, 1 and 2, 3, the splits held up the state's: 83 for 78 us a call at
//     256 slices, 1990 for 1935 at 128.
// Three buffers (two chunks ahead) for the forward bf16 walk: with two the 256
// slices below take 5 us more, a call of N = 128 over 65536 tokens 2267 us for 1945.
//
// A chunk takes 2700 cycles at N = 64, LDS busy for 1120 of them and waiting on
// bank conflicts for 280; 3590, 1540 and 420 at N = 128.  Over 32 chunks, 256
// slices: 42 us (N = 64); over 1024 chunks, 128 slices at N = 128: 1665 us.  The
// first kernel, one workgroup of four wavefronts that loaded and computed in turn,
// took 110 and 4730 us.
//
// K rows lie in LDS in blocks of 8 values whose place is permuted by the row
// (k_block), which keeps both the row-wise and the transposed reads free of
// bank conflicts without padding, as the direct loads need it.
// TRAIN (the gradient's two walks, which run beside each other): no output
// wavefronts, and buffers for one chunk ahead only, so that two workgroups fit on
// a CU at N = 128 too: 79 us for both walks at 256 slices each (N = P = 64, 32
// chunks), where two chunks ahead fit as well and take 81.
template <typename IO, int N, bool TRAIN> struct WalkCfg {
    static constexpr int KP = DeltaPlanes<IO>::io, WP = DeltaPlanes<IO>::wide;
    static constexpr bool DIRECT = KP == 1;           // io values are operands as they are: loads go straight to LDS
    static constexpr int NBUF = DIRECT && !TRAIN ? 3 : 2;
    static constexpr int KB = N / 32, NT = N / 16, TI = (NT + 3) / 4;
    static constexpr int outs = TRAIN ? 0 : 3, waves = 4 + outs + 1;
    // bytes of one buffer (T apart: the gradient has one, and float32 at N = 128,
    // whose planes leave room for one)
    static constexpr int k = 0, f = k + KP * 64 * N * 2, v = f + 5 * 256, buf = v + (DIRECT ? 64 * 32 : 0);
    static constexpr int tsize = kTriBlocks * WP * 1024, TB = TRAIN || (!DIRECT && N == 128) ? 1 : NBUF;
    static constexpr int t = NBUF * buf;
    // then the planes of S, R, d U, U itself, and the rows of O
    static constexpr int ex = t + TB * tsize, s = 0, r = s + WP * KB * 1024, u2 = r + WP * 2048, u = u2 + WP * 2048,
                         o = u + 4096, total = ex + (TRAIN ? u : o + 64 * 16 * (int)sizeof(IO));
    // loads of one chunk by the loader (DIRECT): T, factors, K, V
    static constexpr int loads = kTriBlocks * WP + 2 + 64 * N * 2 / 1024 + 2;
};

// Where block j (8 values) of row t lies in its row.
template <int N> __device__ __forceinline__ int k_block(int t, int j)
{
    if constexpr (N == 32) return j ^ ((t >> 3) & 3);
    else if constexpr (N == 64) return j ^ (((t >> 1) & 1) | (((t >> 3) & 3) << 1));
    else return j ^ ((t & 3) | (((t >> 3) & 3) << 2));
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

// 16 (4) bytes a lane from memory to LDS at base + 16 (4) lane.
__device__ __forceinline__ void to_lds16(char* base, const void* src)
{
    __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)base, 16, 0, 0);
}
__device__ __forceinline__ void to_lds4(char* base, const void* src)
{
    __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)base, 4, 0, 0);
}
// Waits until at most n of this wavefront's memory loads are in flight.
template <int n> __device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}
// And for all of its LDS writes.
template <int n> __device__ __forceinline__ void wait_loads_lds()
{
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
}

// The loader wavefront of a walk: K, the triangle `tri`, the factors and (not
// REV) V of each chunk to LDS, NBUF - 1 steps ahead of their use.  REV: chunks
// from the last to the first.
template <typename IO, int N, bool TRAIN, bool REV>
__device__ __forceinline__ void walk_loader(const DeltaParams& p, char* wlds, const bf16* tri, const DeltaRow& row, int h,
                                            int p0, int nch, int nlast, int lane)
{
    using Cf = WalkCfg<IO, N, TRAIN>;
    constexpr int KP = Cf::KP, WP = Cf::WP, NBUF = Cf::NBUF;
    constexpr bool T1 = Cf::TB == 1;
    const int rs = p.G * N, vs = p.H * p.P;
    const int64_t ci0 = row.slot0 * p.H + h;
    const IO* kp = reinterpret_cast<const IO*>(p.k) + (row.start * p.G + h / (p.H / p.G)) * N;
    const IO* vp = reinterpret_cast<const IO*>(p.v) + (row.start * p.H + h) * p.P + p0;
    // (s: step of the walk)
    auto stage_t = [&](int s, int i0, int i1) {   // blocks i0..i1-1 of the triangle
        const int c = REV ? nch - 1 - s : s;
        char* dst = wlds + Cf::t + (s % Cf::TB) * Cf::tsize;
        const char* src = reinterpret_cast<const char*>(tri + (ci0 + (int64_t)c * p.H) * (kTriBlocks * WP * 512));
#pragma unroll
        for (int i = 0; i < kTriBlocks * WP; ++i)
            if (i >= i0 && i < i1) to_lds16(dst + 1024 * i, src + 1024 * i + 16 * lane);
    };
    // factors, V, K: loads i0..i1-1 of `head`
    constexpr int nk = 64 * N * 2 / 1024, nv = REV ? 0 : 2, head = 2 + nv + nk;
    constexpr int RPL = 512 / N, NR = 64 / RPL;   // K rows of one load; loads of a chunk's K
    // float32 K waits in registers, one more chunk ahead, for its split into
    // planes; `split` also reads the next chunk's row in its place
    RawRow8<IO> raw[Cf::DIRECT ? 1 : NR];
    auto fetch = [&](int s, int i) {
        if constexpr (!Cf::DIRECT) {
            s = s < nch ? s : nch - 1;
            const int c = REV ? nch - 1 - s : s;
            const int end = c == nch - 1 ? nlast - 1 : kDC - 1;
            const int t = RPL * i + lane / (N / 8), j = k_block<N>(t, lane % (N / 8));
            raw[i].load(kp + (int64_t)c * kDC * rs + (t < end ? t : end) * rs + 8 * j, true);
        }
    };
    auto split = [&](int s, int i0, int i1) {
        if constexpr (!Cf::DIRECT) {
            char* buf = wlds + (s % NBUF) * Cf::buf;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if (i < i0 || i >= i1) continue;
                bf16x8 o[KP];
                raw[i].planes(o);
#pragma unroll
                for (int q = 0; q < KP; ++q)
                    *reinterpret_cast<bf16x8*>(buf + Cf::k + q * (64 * N * 2) + 1024 * i + 16 * lane) = o[q];
                fetch(s + 1, i);
            }
        }
    };
    auto stage = [&](int s, int i0, int i1) {
        const int c = REV ? nch - 1 - s : s;
        char* buf = wlds + (s % NBUF) * Cf::buf;
        const int end = c == nch - 1 ? nlast - 1 : kDC - 1;   // last row to read
        const IO* kc = kp + (int64_t)c * kDC * rs;
        const float* fsrc = p.sc + (ci0 + (int64_t)c * p.H) * (kDScal * 64);
        if (i0 == 0) {
            to_lds16(buf + Cf::f, fsrc + 4 * lane);
            to_lds4(buf + Cf::f + 1024, fsrc + 256 + lane);
        }
        if constexpr (Cf::DIRECT) {
#pragma unroll
            for (int i = 0; i < nk; ++i) {
                if (2 + nv + i < i0 || 2 + nv + i >= i1) continue;
                const int t = RPL * i + lane / (N / 8), j = k_block<N>(t, lane % (N / 8));
                to_lds16(buf + Cf::k + 1024 * i, kc + (t < end ? t : end) * rs + 8 * j);
            }
            if (!REV && i0 == 0) {
                const IO* vc = vp + (int64_t)c * kDC * vs;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = 32 * i + lane / 2;
                    to_lds16(buf + Cf::v + 1024 * i, vc + (t < end ? t : end) * vs + 8 * (lane % 2));
                }
            }
        }
    };
    // s_barrier alone: the release of __syncthreads would wait for every load
    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    if (!Cf::DIRECT && nch > 0)
#pragma unroll
        for (int i = 0; i < NR; ++i) fetch(0, i);
#pragma unroll
    for (int s = 0; s < NBUF - 1; ++s)
        if (s < nch) {
            stage(s, 0, head);
            split(s, 0, NR);
            if (s < Cf::TB) stage_t(s, 0, 3 * kTriBlocks);
        }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    barrier();
    for (int s = 0; s < nch; ++s) {
        // a third of the loads (float32: of the splits) beside each stage: a load
        // takes some 30 cycles to issue, all of one chunk longer than a stage
        constexpr int third = (head + 18) / 3;
        constexpr int k1 = Cf::DIRECT && !T1 && third < head ? third : head, t1 = 2 * third > head ? 2 * third - head : 0;
        constexpr int NR1 = NR / 3, NR2 = 2 * NR / 3;
        const bool more = s + NBUF - 1 < nch;
        if (more) {
            stage(s + NBUF - 1, 0, k1);
            if (!Cf::DIRECT) {
                if (!T1) stage_t(s + NBUF - 1, 0, 18);
                asm volatile("" ::: "memory");   // the last loads of a step are rows, for the wait below
                split(s + NBUF - 1, 0, NR1);
            }
        }
        barrier();   // R
        if (!Cf::DIRECT && more) split(s + NBUF - 1, NR1, NR2);
        if (Cf::DIRECT && !T1 && more) {
            if (k1 < head) stage(s + NBUF - 1, k1, head);
            stage_t(s + NBUF - 1, 0, t1);
        }
        barrier();   // U: a single T is free
        if (!T1) {
            if (Cf::DIRECT && more) stage_t(s + NBUF - 1, t1, 18);
            if (!Cf::DIRECT && more) split(s + NBUF - 1, NR2, NR);
        } else if (s + 1 < nch) {
            stage_t(s + 1, 0, 18);
            asm volatile("" ::: "memory");
            if (!Cf::DIRECT && more) split(s + NBUF - 1, NR2, NR);
        }
        asm volatile("" ::: "memory");
        // the next chunk has landed
        constexpr int loads = Cf::loads - (REV ? 2 : 0);
        if (NBUF == 3 && more) wait_loads<loads>();
        else if (!Cf::DIRECT && !T1 && more) wait_loads_lds<2 * NR>();   // (the rows fetched meanwhile)
        else if (!Cf::DIRECT && more) wait_loads_lds<2 * (NR - NR2)>();
        else __builtin_amdgcn_s_waitcnt(0);
        barrier();   // S
    }
}

template <typename IO, int N, bool TRAIN>
__device__ __forceinline__ void delta_walk(const DeltaParams& p, float* Sbuf, float* Ubuf, int64_t bid, char* wlds)
{
    using Cf = WalkCfg<IO, N, TRAIN>;
    constexpr int KP = Cf::KP, WP = Cf::WP, KB = Cf::KB, NT = Cf::NT, TI = Cf::TI, NBUF = Cf::NBUF;

    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the slices of one (row, head) run on one XCD and share its L2
    const int nsl = p.P / 16;
    const int64_t idx = bid >> 3;
    const int64_t unit = (idx / nsl) * 8 + (bid & 7);
    if (unit >= (int64_t)p.rows * p.H) return;
    int b, h;
    delta_unit(p, unit, b, h);
    const int p0 = (int)(idx % nsl) * 16;   // first column
    const DeltaRow row = delta_row(p, b);
    const int64_t rec = TRAIN ? b : delta_record(p, b, tid, 64 * Cf::waves, reinterpret_cast<int*>(wlds));
    const int nch = (int)((row.len + kDC - 1) / kDC);
    const int rs = p.G * N, vs = p.H * p.P;
    const int64_t ci0 = row.slot0 * p.H + h;
    // Rows past the sequence's end read its last row instead: their beta is 0
    // and T's rows there are the identity's, so they write and decay nothing.
    const int nlast = (int)(row.len - (int64_t)(nch - 1) * kDC);   // tokens of the last chunk

    if (wave == Cf::waves - 1) {
        walk_loader<IO, N, TRAIN, false>(p, wlds, p.tf, row, h, p0, nch, nlast, lane);
        return;
    }

    const f32x4 fz = {0.f, 0.f, 0.f, 0.f};
    char* ex = wlds + Cf::ex + 16 * lane;

    if constexpr (!TRAIN)
    if (wave >= 4) {   // output: row tiles 0 and 1, tile 2, tile 3, two of A's blocks each
        // No load depends on a branch: where one might, a wait for the chunk's
        // operands would also wait for those of the chunk after it.
        auto output = [&](auto first_) {
        constexpr bool FIRST = decltype(first_)::value;
        constexpr int TO = FIRST ? 2 : 1;            // row tiles
        const int tile = FIRST ? 0 : wave - 3;       // the first
        const IO* qp = reinterpret_cast<const IO*>(p.q) + (row.start * p.G + h / (p.H / p.G)) * N + 8 * g;
        IO* op = reinterpret_cast<IO*>(p.o) + (row.start * p.H + h) * p.P + p0;
        IO* so = reinterpret_cast<IO*>(wlds + Cf::ex + Cf::o) + (FIRST ? 0 : 16 * tile) * 16;   // this wave's rows, tile by tile
        RawRow8<IO> q[TO][KB];
        f32x4 a[2][2];   // [block][half]
        bf16x8 a8[2][WP], u8[2][WP];
        f32x4 acc[TO], out[TO];
        auto load = [&](int c) {
            c = c < nch ? c : nch - 1;
            const int end = c == nch - 1 ? nlast - 1 : kDC - 1;
            const IO* qc = qp + (int64_t)c * kDC * rs;
#pragma unroll
            for (int i = 0; i < TO; ++i) {
                const int t = tile_row(tile + i, l) < end ? tile_row(tile + i, l) : end;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) q[i][kb].load(qc + t * rs + 32 * kb, true);
            }
        };
        auto load_a = [&](int c) {   // blocks (0, 0) and (1, 0), or (tile, 0) and (tile, 1)
            c = c < nch ? c : nch - 1;
            const float* src = p.af + (ci0 + (int64_t)c * p.H) * (int64_t)kTriValues + 4 * lane;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    a[i][j] = *reinterpret_cast<const f32x4*>(src + (FIRST ? low_block(i, 0) : low_block(tile, i)) * 512 + 256 * j);
        };
        auto split_a = [&](int i) { planes8<WP>(a[i][0], a[i][1], a8[i]); };
        auto split_u = [&]() {
#pragma unroll
            for (int kb = 0; kb < (FIRST ? 1 : 2); ++kb)
                planes8<WP>(*reinterpret_cast<const f32x4*>(ex + Cf::u + 2 * kb * 1024),
                            *reinterpret_cast<const f32x4*>(ex + Cf::u + (2 * kb + 1) * 1024), u8[kb]);
        };
        auto add_u = [&]() {   // + A U
#pragma unroll
            for (int i = 0; i < TO; ++i) out[i] = acc[i];
            if constexpr (FIRST) {
                mma_tiles<2, WP, WP, WP>(a8, u8[0], out);
            } else {
                mma_planes<WP, WP, WP>(a8[0], u8[0], out[0]);
                mma_planes<WP, WP, WP>(a8[1], u8[1], out[0]);
            }
        };
        auto store = [&](int c) {   // through LDS: 16 bytes of a row to a lane, not 2
#pragma unroll
            for (int i = 0; i < TO; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) so[(16 * i + 4 * g + r) * 16 + l] = from_f32<IO>(out[i][r]);
            wave_order();
            const int nv = c == nch - 1 ? nlast : kDC;
            IO* oc = op + (int64_t)c * kDC * vs;
            constexpr int per = 16 / sizeof(IO), lpr = 16 / per, rows = 64 / lpr;   // values to a lane, lanes to a row, rows to a store
#pragma unroll
            for (int i = 0; i < (16 * TO + rows - 1) / rows; ++i) {
                const int m = rows * i + lane / lpr, j = lane % lpr;
                const int t = tile_row(tile + (m >> 4), m & 15);
                if (m < 16 * TO && t < nv)
                    *reinterpret_cast<uint4*>(oc + t * vs + per * j) = *reinterpret_cast<const uint4*>(so + m * 16 + per * j);
            }
            wave_order();
        };
        if (nch > 0) {
            load(0);
            load_a(0);
        }
        __syncthreads();
        for (int c = 0; c < nch; ++c) {
            if (c > 0) {
                add_u();
                store(c - 1);
            }
            __syncthreads();   // R
#pragma unroll
            for (int i = 0; i < TO; ++i) acc[i] = fz;
            f32x4 fo[TO];
#pragma unroll
            for (int i = 0; i < TO; ++i)
                fo[i] = *reinterpret_cast<const f32x4*>(wlds + (c % NBUF) * Cf::buf + Cf::f + 4 * (192 + tile_row(tile + i, 4 * g)));
            split_a(0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8 s8[WP], q8[TO][KP];
#pragma unroll
                for (int j = 0; j < WP; ++j) s8[j] = *reinterpret_cast<const bf16x8*>(ex + Cf::s + (j * KB + kb) * 1024);
#pragma unroll
                for (int i = 0; i < TO; ++i) q[i][kb].planes(q8[i]);
                mma_tiles<TO, KP, WP, WP>(q8, s8, acc);
            }
#pragma unroll
            for (int i = 0; i < TO; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] *= fo[i][r];
            load(c + 1);
            __syncthreads();   // U
            split_u();
            split_a(1);
            load_a(c + 1);
            __syncthreads();   // S
        }
        if (nch > 0) {
            add_u();
            store(nch - 1);
        }
        };
        if (wave == 4) output(std::true_type());
        else output(std::false_type());
        return;
    }

    // state: wave w has tile w of R and U and tiles w, w + 4 of the state, rows
    // tile_row(tile, 4 g + r), column l
    const int w = wave & 3;
    const int tr0 = 32 * (w >> 1) + 4 * (w & 1) + 8 * g;   // first row of tile w in this lane
    const int nb = (w >> 1) + 1;                           // 32-token blocks that tile w of T spans
    const int half = 8 * (w & 1);                          // its place in an operand's 16 bytes
    const int col = p0 + l;
    f32x4 S[TI];
    const float* hin = p.h_in != nullptr && rec >= 0 ? p.h_in + (rec * p.H + h) * (int64_t)(N * p.P) + col : nullptr;
    if (!TRAIN && p.carry_in != nullptr) hin = p.carry_in + ((int64_t)b * p.H + h) * (int64_t)(N * p.P) + col;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            S[i][r] = hin != nullptr && w + 4 * i < NT ? hin[(tr0 + 64 * i + r) * p.P] : 0.f;
            if (rec == -2) S[i][r] = __builtin_nanf("");   // the record belongs to an earlier row
        }
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

    // V of float32 calls comes from memory one chunk ahead, of bf16 calls from LDS
    const IO* vp = reinterpret_cast<const IO*>(p.v) + (row.start * p.H + h) * p.P + col;
    float vnext[4];
    auto load_v = [&](int c) {
        if constexpr (!Cf::DIRECT) {
            const int end = c == nch - 1 ? nlast - 1 : kDC - 1;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                vnext[r] = to_f32(vp[(int64_t)c * kDC * vs + (tr0 + r < end ? tr0 + r : end) * vs]);
        }
    };
    if (nch > 0) load_v(0);
    __syncthreads();

    for (int c = 0; c < nch; ++c) {
        const char* buf = wlds + (c % NBUF) * Cf::buf;
        const int64_t ci = ci0 + (int64_t)c * p.H;
        if (TRAIN) {
            float* sd = Sbuf + ci * N * p.P + col;
#pragma unroll
            for (int i = 0; i < TI; ++i)
                if (w + 4 * i < NT)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sd[(tr0 + 64 * i + r) * p.P] = S[i][r];
        }
        // R = beta V - sp (K S)
        const float* f = reinterpret_cast<const float*>(buf + Cf::f) + tr0;
        const char* tb = wlds + Cf::t + (c % Cf::TB) * Cf::tsize + 16 * lane;
        bf16x8 t8[2][WP];   // T's rows, read beside the other operands
        const f32x4 fu = *reinterpret_cast<const f32x4*>(f + 128);
        const float eL = *reinterpret_cast<const float*>(buf + Cf::f + 1024 + 4 * lane);
        f32x4 P = fz;
        {
            const int t = tile_row(w, l);
            bf16x8 k8[KB][KP], s8[KB][WP];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int j = 0; j < WP; ++j) s8[kb][j] = *reinterpret_cast<const bf16x8*>(ex + Cf::s + (j * KB + kb) * 1024);
#pragma unroll
                for (int j = 0; j < KP; ++j)
                    k8[kb][j] = *reinterpret_cast<const bf16x8*>(buf + Cf::k + j * (64 * N * 2) + t * (2 * N) +
                                                                 16 * k_block<N>(t, 4 * kb + g));
            }
            const f32x4 fb = *reinterpret_cast<const f32x4*>(f), fp = *reinterpret_cast<const f32x4*>(f + 64);
            float v[4];
            if constexpr (Cf::DIRECT) {
                const bf16x4 x = lds_read_tr4(reinterpret_cast<const bf16*>(buf + Cf::v) +
                                              (tr0 + (l >> 2)) * 16 + 4 * (l & 3));
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = (float)x[r];
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = vnext[r];
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < WP; ++j)
                    t8[kb][j] = *reinterpret_cast<const bf16x8*>(tb + (low_block(w, kb < nb ? kb : 0) * WP + j) * 1024);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) mma_planes<KP, WP, WP>(k8[kb], s8[kb], P);
            f32x4 R;
#pragma unroll
            for (int r = 0; r < 4; ++r) R[r] = fb[r] * v[r] - fp[r] * P[r];
            bf16x4 o[WP];
            to_planes4<WP>(R, o);
#pragma unroll
            for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x4*>(ex + Cf::r + (2 * j + (w >> 1)) * 1024 + half) = o[j];
        }
        if (c + 1 < nch) load_v(c + 1);
        __syncthreads();
        // U = T R
        f32x4 U = fz;
        bf16x8 r8[2][WP];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb < nb)
#pragma unroll
                for (int j = 0; j < WP; ++j) r8[kb][j] = *reinterpret_cast<const bf16x8*>(ex + Cf::r + (2 * j + kb) * 1024);
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
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb < nb) mma_planes<WP, WP, WP>(t8[kb], r8[kb], U);
        {
            f32x4 u2;
#pragma unroll
            for (int r = 0; r < 4; ++r) u2[r] = fu[r] * U[r];
            bf16x4 o[WP];
            to_planes4<WP>(u2, o);
#pragma unroll
            for (int j = 0; j < WP; ++j) *reinterpret_cast<bf16x4*>(ex + Cf::u2 + (2 * j + (w >> 1)) * 1024 + half) = o[j];
            if constexpr (!TRAIN) {
                *reinterpret_cast<f32x4*>(ex + Cf::u + w * 1024) = U;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) Ubuf[(ci * 64 + tr0 + r) * p.P + col] = U[r];
            }
        }
        __syncthreads();
        // S <- e^G_last S + K^T (d U)
        f32x4 acc[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) acc[i] = fz;
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
    float* ho = !TRAIN && p.h_out != nullptr && rec >= 0 ? p.h_out + (rec * p.H + h) * (int64_t)(N * p.P) + col : nullptr;
    if (!TRAIN && p.carry_out != nullptr) ho = p.carry_out + ((int64_t)b * p.H + h) * (int64_t)(N * p.P) + col;
    if (ho != nullptr) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (w + 4 * i < NT)
#pragma unroll
                for (int r = 0; r < 4; ++r) ho[(tr0 + 64 * i + r) * p.P] = S[i][r];
    }
}

template <typename IO, int N>
__global__ __launch_bounds__(64 * 8) void delta_walk_kernel(const DeltaParams p)
{
    extern __shared__ __attribute__((aligned(16))) char wlds[];
    delta_walk<IO, N, false>(p, nullptr, nullptr, blockIdx.x, wlds);
}

// Lets `kern` have `bytes` of LDS on the current device, once on each (`done`:
// a bit per device, one word per kernel).
template <typename F> hipError_t delta_allow_lds(F* kern, size_t bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;   // (past 64: each time)
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    else (void)hipGetLastError();
    return e;
}

template <typename IO, int N>
hipError_t launch_delta_walk(const DeltaParams& p, hipStream_t stream)
{
    using Cf = WalkCfg<IO, N, false>;
    auto* const kern = &delta_walk_kernel<IO, N>;
    static_assert(Cf::total <= 160 * 1024, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    const hipError_t attr = delta_allow_lds(kern, Cf::total, done);
    if (attr != hipSuccess) return attr;
    const int64_t blocks = ((int64_t)p.rows * p.H + 7) / 8 * 8 * (p.P / 16);
    const size_t lds = Cf::total;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * Cf::waves), lds, stream, p);
    return hipGetLastError();
}

}  // namespace m3
