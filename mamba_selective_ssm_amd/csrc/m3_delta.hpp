// Gated delta rule: what its translation units share.
//
//   S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - (a_t S_{t-1})^T k_t),
//   o_t = scale S_t^T q_t,           a_t = exp(g_t)
//
// Chunked form, 64 tokens to a chunk.  With G_t the running sum of g inside the
// chunk, S0 the state before it, e = exp(G), d_t = exp(G_last - G_t) and
// D_ij = exp(G_i - G_j) for j <= i:
//   (I + M) U = beta (V - e K S0),  M_ij = beta_i D_ij k_i.k_j  (j < i)
//   O  = scale (e Q S0 + (D o Q K^T) U)
//   S1 = exp(G_last) S0 + K^T (d U)
// T = (I + M)^-1 does not depend on the state, so it is made for all chunks at
// once; what is left for the walk over a sequence's chunks is three products a
// chunk, each of them independent for every column of V.
//
// Matrix cores multiply bf16 operands here.  A float32 operand is the sum of
// up to three bf16 values ("planes": its rounding, the rounding of what that
// left, and once more), 24 bits together, and a product of two such operands
// adds the plane products that float32 can still see: 3 where one side is an
// exact bf16 value, 6 where both have three planes.  At 16x16x32 that is 48
// and 96 cycles against 256 of the float32 instructions for the same product.
// Every product's operands are held so, the output's too: a bf16 output is one
// rounding of a value as exact as float32's (with two planes for S, U and A there
// its error before that rounding was 2.5e-6 of the outputs' size, for 1e-7 now).
#pragma once

#include "m3_device.hpp"
#include "m3_internal.hpp"

namespace m3 {

constexpr int kDC = 64;        // tokens per chunk
constexpr int kDScal = 8;      // per-token factor rows that the chunk kernel leaves

struct DeltaParams {
    const void *q, *k, *v;
    const float *g, *beta;
    const float *h_in;
    void *o;
    float *h_out;
    const int* cu;         // [rows + 1] packed-sequence offsets, or NULL
    const int* slots;      // [rows] record of each row, or NULL (row b: record b)
    int64_t nslots;        // records that h_in / h_out hold
    int64_t L;             // tokens per row; packed: tokens in all
    int64_t max_len;       // longest row
    int rows, H, G;        // batch rows or sequences, heads, q/k head groups
    int N, P;
    float scale, eps;
    int l2norm;
    int nc;                // chunks of the longest row, or of the part
    int64_t places;        // packed rows far shorter than max_len: chunk slots, which the chunks' kernels go by; else 0
    int64_t from, count;   // the part of each row that a launch works on, in chunks (count 0: all of it)
    const float* carry_in; // [rows][H][N][P] state before that part where it is not the row's first, else NULL
    float* carry_out;      // and behind it where it is not the last
    // workspace, one entry per (chunk slot, head)
    bf16* tf;              // T in operand order
    float* af;             // scale D o Q K^T in operand order
    float* sc;             // [kDScal][64] per-token factors
    int* order;            // [rows] packed rows, most chunks first (NULL: as they stand)
};

// Gradient: what the kernels add to the above.
struct DeltaBwdParams {
    DeltaParams f;
    const void* dout;
    const float* dh_out;
    float *dq, *dk, *dv, *dg, *dbeta, *dh_in;
    float* S;              // [chunk][N][P] state before each chunk
    float* dS;             // [chunk][N][P] adjoint of the state after each chunk
    float* U;              // [chunk][64][P]
    float* dR;             // [chunk][64][P]
    float *dqe, *dke;      // [token][H][N] per-head gradients where heads share q and k, else dq and dk
};

hipError_t launch_delta_fwd(const DeltaParams& p, int io_dtype, hipStream_t stream);
hipError_t launch_delta_bwd_f32(const DeltaBwdParams& p, hipStream_t stream);
hipError_t launch_delta_bwd_bf16(const DeltaBwdParams& p, hipStream_t stream);
hipError_t launch_delta_step(const DeltaParams& p, int io_dtype, hipStream_t stream);

constexpr bool delta_supported(int64_t N, int64_t P, int io_dtype)
{
    return (N == 32 || N == 64 || N == 128) && P >= 32 && P <= 128 && P % 32 == 0 && (io_dtype == 0 || io_dtype == 1);
}

// Long prefills whose walk leaves CUs idle are walked in parts, each beside the
// chunk matrices of the next, which the walk then reads out of the caches.  Whole
// calls, us, at once / in parts, P = 64, bf16: 65536 tokens, 128 slices, N = 128:
// 2105 / 1945; 16384: 553 / 500; 8192: 272 / 246; 4096: 128 / 125; N = 64, 65536
// tokens, 32 slices: 1598 / 1215, 64: 1710 / 1382; 8192, 192: 302 / 249.  At 256
// slices no CU is left over and it goes either way: N = 64, 32768 tokens: 1208 /
// 1133, 8192: 327 / 297; N = 128, 16384: 679 / 707, 8192: 353 / 359.
// A part is as many chunks as leave its rows and matrices in the caches together
// with the next one's, about 1024 chunks and heads in bf16: 32 heads, N = 128,
// parts of 16 / 32 / 48 / 64 / 128 chunks: 1927 / 1949 / 2005 / 2024 / 2024 us;
// float32, 16 heads, N = 64, 16384 tokens: 646 / 606 / 607 / 630 / 721 (at once:
// 731).  It has to be long beside a launch and the walk's first loads, 32 chunks
// at least: 16 heads, N = 64, 16384 tokens: 375 / 342 / 330 / 311 / 311 (at once:
// 313).  Calls of two such parts or less lie in the caches as they are: 1 head, N
// = 64, 32768 tokens: 542 / 573; 16 heads, float32, 4096: 162 / 167.
constexpr int64_t delta_part_size(int io_dtype) { return io_dtype == 0 ? 512 : 1024; }
constexpr int64_t delta_part(int64_t units, int io_dtype)
{
    const int64_t n = delta_part_size(io_dtype) / (units > 0 ? units : 1);
    return n < 32 ? 32 : n > 64 ? 64 : n;
}
constexpr bool delta_in_parts(int64_t units, int64_t nc, int64_t P, int io_dtype)
{
    return units * (P / 16) <= 192 && nc >= 2 * delta_part(units, io_dtype) && units * nc > 2 * delta_part_size(io_dtype);
}

// Planes of float32 operands, and of the io type's own values.
template <typename IO> struct DeltaPlanes;
template <> struct DeltaPlanes<bf16> { static constexpr int io = 1, wide = 3; };
template <> struct DeltaPlanes<float> { static constexpr int io = 3, wide = 3; };

// Row m of 16 x 16 tile i, for the tokens of a chunk and for the rows of the
// state alike.  A result tile leaves rows 4 g + r (r = 0..3) in lane (l, g);
// with this order the tiles 2 kb and 2 kb + 1 leave rows 32 kb + 8 g .. + 7
// there: the eight K values of the second operand of the next product.  So a
// wavefront feeds a product's result to the next one in its own registers.
__host__ __device__ constexpr int tile_row(int i, int m) { return 32 * (i >> 1) + 8 * (m >> 2) + 4 * (i & 1) + (m & 3); }

// Operand blocks of a lower triangular 64 x 64 matrix, 16 rows (of tile w) x 32
// columns each, in the order (0,0) (1,0) (2,0) (3,0) (2,1) (3,1) of (w, kb).
constexpr int kTriBlocks = 6;
__host__ __device__ constexpr int low_block(int w, int kb) { return w + 2 * kb; }

constexpr size_t kTriValues = (size_t)kTriBlocks * 512;

// What a wavefront's lanes have written to LDS before is there for all its
// lanes after: its LDS instructions run in order, so only the compiler's order
// has to be held.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Where a row's tokens lie: its first token row, its length, its first chunk
// slot.  Offsets are clamped into the arrays and lengths to max_len, so that
// wrong ones give wrong results and no access outside.
struct DeltaRow {
    int64_t start, len, slot0;
};
__device__ __forceinline__ DeltaRow delta_row(const DeltaParams& p, int b)
{
    DeltaRow r;
    if (p.cu == nullptr) {
        r.start = (int64_t)b * p.L;
        r.len = p.L;
        r.slot0 = (int64_t)b * ((p.L + kDC - 1) / kDC);
    } else {
        int64_t s = p.cu[b], e = p.cu[b + 1];
        s = s < 0 ? 0 : (s > p.L ? p.L : s);
        e = e < s ? s : (e > p.L ? p.L : e);
        r.start = s;
        r.len = e - s < p.max_len ? e - s : p.max_len;
        // floor(a + b) + 1 >= floor(a) + ceil(b): no two rows share a slot
        r.slot0 = s / kDC + b;
    }
    if (p.count > 0) {
        const int64_t left = r.len - p.from * kDC;
        r.start += left > 0 ? p.from * kDC : 0;
        r.slot0 += p.from;
        r.len = left < 0 ? 0 : left < p.count * kDC ? left : p.count * kDC;
    }
    return r;
}

// Row and chunk of the bc'th of a launch over chunks: nc to a row, or by chunk
// slots where most of those would be empty (more than twice as many: a bound far
// above the lengths, such as the default one) or too many for a launch.  Rows'
// first slots ascend, every row has one at least.  A slot of no row gets a chunk
// behind its end.  300 rows of 60000 tokens in all, 16 heads, N = P = 64, bounded
// by 60000: 470 us for 1576 (by the longest: 476); the gradient, 30000 tokens: 1219
// for 5002 (1178).
inline int64_t delta_chunk_count(const DeltaParams& p) { return p.places > 0 ? p.places : (int64_t)p.rows * p.nc; }
__device__ __forceinline__ void delta_place(const DeltaParams& p, int bc, int& b, int& c)
{
    if (p.places == 0) {
        c = bc % p.nc;
        b = bc / p.nc;
        return;
    }
    auto slot0 = [&](int row) {
        const int64_t s = p.cu[row];
        return (int)((s < 0 ? 0 : s > p.L ? p.L : s) / kDC) + row;
    };
    int lo = 0, hi = p.rows;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (slot0(mid) <= bc) lo = mid;
        else hi = mid;
    }
    b = lo;
    c = bc - slot0(lo);
    if (c < 0) c = 1 << 30;
}

// Row and head of a walk's workgroup.  The rows with the most chunks come first:
// a CU whose last workgroup is a long one holds up the call.  13 sequences of 7
// to 40 chunks, 32 heads, N = P = 128: calls of 552 us for 586 one at a time; the
// gradient, 7 sequences of 4099 tokens in all, 16 heads: 244 for 254.
__device__ __forceinline__ void delta_unit(const DeltaParams& p, int64_t unit, int& b, int& h)
{
    int64_t b64, h64;
    split_bh(unit, p.H, b64, h64);
    b = p.order != nullptr ? p.order[b64] : (int)b64;
    h = (int)h64;
}

// Called by one wavefront: puts row b at its place in the order.
__device__ __forceinline__ void delta_rank(const DeltaParams& p, int b, int lane)
{
    const int64_t mine = (delta_row(p, b).len + kDC - 1) / kDC;
    int before = 0;
    for (int i = lane; i < p.rows; i += 64) {
        const int64_t n = (delta_row(p, i).len + kDC - 1) / kDC;
        before += n > mine || (n == mine && i < b) ? 1 : 0;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) before += __shfl_xor(before, m);
    if (lane == 0) p.order[before] = b;
}

// The record of row b: its index, -1 for none (a slot outside the pool), -2
// where an earlier row names the same slot.  Called by whole workgroups; lane
// ids run over [0, nt).
__device__ __forceinline__ int64_t delta_record(const DeltaParams& p, int b, int tid, int nt, int* flag)
{
    if (p.slots == nullptr) return b;
    const int s = p.slots[b];
    if (s < 0 || s >= p.nslots) return -1;
    bool seen = false;
    for (int i = tid; i < b; i += nt) seen |= p.slots[i] == s;
    if (tid == 0) *flag = 0;
    __syncthreads();
    if (seen) *flag = 1;
    __syncthreads();
    const int twice = *flag;
    __syncthreads();
    return twice ? -2 : s;
}

// A bf16 pair in a scalar register.  (As a constant, (-1, 0) would become the
// instruction's inline -1.0, which it takes for both halves.)
__device__ __forceinline__ bf16x2 pair_of(unsigned bits)
{
    asm("" : "+s"(bits));
    return __builtin_bit_cast(bf16x2, bits);
}

// Two values as sums of bf16 planes: each plane is the rounding of what the
// ones before it left, one conversion for both.
typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
template <int PL> __device__ __forceinline__ void to_planes2(float x, float y, bf16x2 (&o)[PL])
{
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        o[i] = __builtin_convertvector(f32x2{x, y}, bf16x2);
        if (i + 1 < PL) {
            // x - o[0], y - o[1], one instruction each without unpacking
            x = __builtin_amdgcn_fdot2_f32_bf16(o[i], pair_of(0x0000bf80u), x, false);
            y = __builtin_amdgcn_fdot2_f32_bf16(o[i], pair_of(0xbf800000u), y, false);
        }
    }
}
template <int PL> __device__ __forceinline__ void to_planes4(const f32x4& x, bf16x4 (&o)[PL])
{
    bf16x2 a[PL], b[PL];
    to_planes2<PL>(x[0], x[1], a);
    to_planes2<PL>(x[2], x[3], b);
#pragma unroll
    for (int i = 0; i < PL; ++i) o[i] = bf16x4{a[i][0], a[i][1], b[i][0], b[i][1]};
}

// acc[i] += a[i] b, all as planes; products whose planes lie LIM or more apart
// are below what LIM planes hold.  Small ones first.
template <int T, int PA, int PB, int LIM>
__device__ __forceinline__ void mma_tiles(const bf16x8 (&a)[T][PA], const bf16x8 (&b)[PB], f32x4* acc)
{
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < PB)
#pragma unroll
                for (int t = 0; t < T; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][i], b[j], acc[t], 0, 0, 0);
        }
}
template <int PA, int PB, int LIM>
__device__ __forceinline__ void mma_planes(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], f32x4& acc)
{
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < PB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc, 0, 0, 0);
        }
}

__device__ __forceinline__ bf16x8 join8(const bf16x4& a, const bf16x4& b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The same in three planes by cutting off after 8 and 16 bits: each plane is the
// upper half of what those before it left.  More instructions than planes8, of a
// kind that the state waves beside do not wait for: delta_wide's output waves
// with planes8 / this: 166 / 157 us (N = 64, P = 96, 96 rows and heads, 2048
// tokens); delta_walk's, whose time is the way from LDS to the product: 80 / 82.5
// (N = P = 64, 64 of them).
__device__ __forceinline__ void cut8(const f32x4& a, const f32x4& b, bf16x8 (&o)[3])
{
    typedef __attribute__((__vector_size__(4 * sizeof(unsigned)))) unsigned u32x4;
    u32x4 r[3];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float x = e < 4 ? a[e & 3] : b[e & 3], y = e < 4 ? a[(e & 3) + 1] : b[(e & 3) + 1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const unsigned ux = __builtin_bit_cast(unsigned, x), uy = __builtin_bit_cast(unsigned, y);
            r[i][e / 2] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
            if (i < 2) {
                x -= __builtin_bit_cast(float, ux & 0xffff0000u);
                y -= __builtin_bit_cast(float, uy & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) o[i] = __builtin_bit_cast(bf16x8, r[i]);
}

template <int PL> __device__ __forceinline__ void planes8(const f32x4& a, const f32x4& b, bf16x8 (&o)[PL])
{
    bf16x4 x[PL], y[PL];
    to_planes4<PL>(a, x);
    to_planes4<PL>(b, y);
#pragma unroll
    for (int i = 0; i < PL; ++i) o[i] = join8(x[i], y[i]);
}

__device__ __forceinline__ bf16x8 zero8()
{
    bf16x8 z;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = (bf16)0.0f;
    return z;
}

// 8 contiguous io values as planes; zeros where !ok (nothing is read).
template <typename IO> struct RawRow8;
template <> struct RawRow8<bf16> {
    bf16x8 v;
    __device__ __forceinline__ void load(const bf16* p, bool ok) { v = ok ? *reinterpret_cast<const bf16x8*>(p) : zero8(); }
    __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
    __device__ __forceinline__ void planes(bf16x8 (&o)[1]) const { o[0] = v; }
};
template <> struct RawRow8<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p, bool ok)
    {
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
        a = ok ? *reinterpret_cast<const f32x4*>(p) : z;
        b = ok ? *reinterpret_cast<const f32x4*>(p + 4) : z;
    }
    __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
    template <int PL> __device__ __forceinline__ void planes(bf16x8 (&o)[PL]) const
    {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            bf16x2 t[PL];
            to_planes2<PL>(get(e), get(e + 1), t);
#pragma unroll
            for (int i = 0; i < PL; ++i) { o[i][e] = t[i][0]; o[i][e + 1] = t[i][1]; }
        }
    }
};

}  // namespace m3
