// Pools of state records: copy, fork, compact and free slots.
//
// A record is one slot of each of a pool's arrays.  The moves read and write
// each moved byte once and are bound by memory; a workgroup moves one piece
// (16 KiB) of one record, 64 bytes a thread with all its loads in flight.
// Which records move where is decided on the device, so none of these calls
// waits for the host: a launch covers the most moves there can be, and
// workgroups without one leave at once.  Copies of 105 MB run at 4.5 TB/s, a
// compaction that moves 136 MB at 4.9 (a copy of 4 GiB: 4.7); small calls are
// bound by their launches (a fork of 8 records: 14.6 us, two launches and their
// binding).  A copy of very many records is bound by its check: every workgroup
// reads all pairs to find whether its own is the last for its slot, pairs^2 reads
// per piece out of the caches: 4000 records of 256 KiB take 479 us (torch's copy of
// the arrays: 403), 16384 of them 3.5 ms (1.9), 10^5 of 16 KiB 4.0 ms (0.7).
#include "m3_pool.hpp"

namespace m3 {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(unsigned)))) unsigned u32x4;

template <typename T>
__device__ __forceinline__ void move_piece(char* d, const char* s, int64_t bytes)
{
    const int64_t cnt = bytes / (int64_t)sizeof(T);
    const T* sp = reinterpret_cast<const T*>(s);
    T* dp = reinterpret_cast<T*>(d);
    for (int64_t i0 = threadIdx.x; i0 < cnt; i0 += 1024) {
        T t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + 256 * j < cnt) t[j] = sp[i0 + 256 * j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + 256 * j < cnt) dp[i0 + 256 * j] = t[j];
    }
}
template <typename T>
__device__ __forceinline__ void clear_piece(char* d, int64_t bytes)
{
    const int64_t cnt = bytes / (int64_t)sizeof(T);
    T* dp = reinterpret_cast<T*>(d);
    for (int64_t i = threadIdx.x; i < cnt; i += 256) dp[i] = T{};
}

// d == nullptr: nothing; s == nullptr: zeros.
__device__ __forceinline__ void move_bytes(char* d, const char* s, int64_t bytes, int unit)
{
    if (s == nullptr) {
        switch (unit) {
        case 16: clear_piece<u32x4>(d, bytes); break;
        case 4: clear_piece<unsigned>(d, bytes); break;
        case 2: clear_piece<unsigned short>(d, bytes); break;
        default: clear_piece<unsigned char>(d, bytes);
        }
        return;
    }
    switch (unit) {
    case 16: move_piece<u32x4>(d, s, bytes); break;
    case 4: move_piece<unsigned>(d, s, bytes); break;
    case 2: move_piece<unsigned short>(d, s, bytes); break;
    default: move_piece<unsigned char>(d, s, bytes);
    }
}

struct Piece {
    int a;            // array
    int64_t off, len; // bytes of the record's part of it
};
__device__ __forceinline__ Piece piece_of(const PoolParams& p, int j)
{
    Piece r;
    r.a = 0;
    for (int i = 1; i < p.n; ++i)
        if (j >= p.piece0[i]) r.a = i;
    r.off = (int64_t)(j - p.piece0[r.a]) * kPoolPiece;
    const int64_t left = p.row[r.a] - r.off;
    r.len = left < kPoolPiece ? left : kPoolPiece;
    return r;
}

// One piece of pair `pair`'s record.  As if every source were read before
// any slot is written, and the last pair of those that name one slot wins:
//   - a pair with a later one for its slot moves nothing;
//   - in place, a source that is some other pair's slot is staged in the
//     workspace by the first launch (STAGE) and read from there by the second.
// All workgroups of a pair find the same answer from the index arrays alone.
enum { kMove = 0, kStage = 1, kFinish = 2 };
template <int MODE>
__global__ __launch_bounds__(256) void pool_copy_kernel(const PoolParams p, const int* src, const int* dst, int n)
{
    __shared__ int flags[2];
    const int np = p.piece0[p.n];
    const int pair = blockIdx.x / np;
    const int s = src[pair], d = dst[pair];
    if (s >= p.src_slots || d < 0 || d >= p.dst_slots) return;
    if (MODE != kMove && s == d) return;
    if (threadIdx.x < 2) flags[threadIdx.x] = 0;
    __syncthreads();
    bool later = false, staged = false;
    for (int i = threadIdx.x; i < n; i += 256) {
        const int di = dst[i];
        const bool real = src[i] < p.src_slots && di >= 0;
        later |= i > pair && real && di == d;
        if (MODE != kMove) staged |= i != pair && real && di == s;
    }
    if (later) flags[0] = 1;
    if (staged) flags[1] = 1;
    __syncthreads();
    if (flags[0]) return;
    const bool st = flags[1] != 0;
    const Piece q = piece_of(p, blockIdx.x - pair * np);
    const char* from = s < 0 ? nullptr : p.src[q.a] + (int64_t)s * p.row[q.a] + q.off;
    char* to = p.dst[q.a] + (int64_t)d * p.row[q.a] + q.off;
    if (MODE != kMove) {
        char* w = p.ws + (int64_t)pair * p.ws_row + p.ws_off[q.a] + q.off;
        if (MODE == kStage) {
            if (!st) return;
            to = w;
        } else if (st) {
            from = w;
        }
    }
    move_bytes(to, from, q.len, p.unit[q.a]);
}

// Pairs that an earlier kernel of the call has listed: sources and slots
// disjoint, entries below zero left out.
__global__ __launch_bounds__(256) void pool_move_kernel(const PoolParams p, const int* src, const int* dst,
                                                        const int* npairs)
{
    const int np = p.piece0[p.n];
    const int pair = blockIdx.x / np;
    if (npairs != nullptr && pair >= *npairs) return;
    const int s = src[pair], d = dst[pair];
    if (d < 0) return;
    const Piece q = piece_of(p, blockIdx.x - pair * np);
    const char* from = s < 0 ? nullptr : p.src[q.a] + (int64_t)s * p.row[q.a] + q.off;
    move_bytes(p.dst[q.a] + (int64_t)d * p.row[q.a] + q.off, from, q.len, p.unit[q.a]);
}

// Rank of this thread's flag among the workgroup's 1024, and their number.
__device__ __forceinline__ int block_rank(bool f, int* sums, int& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const unsigned long long m = __ballot(f);
    const int below = __popcll(m & ((1ull << lane) - 1));
    __syncthreads();
    if (lane == 0) sums[w] = __popcll(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < 16; ++i) {
        const int v = sums[i];
        before += i < w ? v : 0;
        total += v;
    }
    return before + below;
}

// The lowest free slots for the parents that have a record, in their order.
__global__ __launch_bounds__(1024) void pool_fork_plan(const int* live, int* live_out, int64_t slots, const int* parents,
                                                       int* children, int* list, int64_t n)
{
    __shared__ int sums[16];
    int want = 0, tot;
    for (int64_t i0 = 0; i0 < n; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        bool ok = false;
        if (i < n) {
            const int s = parents[i];
            ok = s < 0 || (s < slots && live[s] != 0);
            children[i] = -1;
        }
        const int r = block_rank(ok, sums, tot);
        if (ok) list[want + r] = (int)i;
        want += tot;
    }
    __syncthreads();
    int got = 0;
    for (int64_t i0 = 0; i0 < slots; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        const int lv = i < slots ? live[i] : 1;
        const int r = block_rank(i < slots && lv == 0, sums, tot);
        if (i < slots) {
            const bool taken = lv == 0 && got + r < want;
            if (taken) children[list[got + r]] = (int)i;
            live_out[i] = taken ? 1 : lv;
        }
        got += tot;
    }
}

// Live records past the front go, in order, to the front's free slots.
// list: [0] their number, then the slots they leave, then those they get
// (half the slots each).
__global__ __launch_bounds__(1024) void pool_compact_plan(const int* live, int* live_out, int64_t slots, int* new_slot,
                                                          int* count, int* list)
{
    __shared__ int sums[16];
    int n = 0, tot;
    for (int64_t i0 = 0; i0 < slots; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        block_rank(i < slots && live[i] != 0, sums, tot);
        n += tot;
    }
    int* from = list + 1;
    int* to = from + slots / 2;
    int nf = 0, nt = 0;
    for (int64_t i0 = 0; i0 < slots; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        const bool on = i < slots && live[i] != 0;
        const int rf = block_rank(on && i >= n, sums, tot);
        if (on && i >= n) from[nf + rf] = (int)i;
        nf += tot;
        const bool hole = i < n && !on;
        const int rt = block_rank(hole, sums, tot);
        if (hole) to[nt + rt] = (int)i;
        nt += tot;
        if (i < slots) {
            if (!(on && i >= n)) new_slot[i] = on ? (int)i : -1;
            if (live_out != nullptr) live_out[i] = i < n ? 1 : 0;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nf; i += 1024) new_slot[from[i]] = to[i];
    if (threadIdx.x == 0) {
        list[0] = nf;
        if (count != nullptr) *count = n;
    }
}

__global__ __launch_bounds__(256) void pool_free_kernel(int* live, int64_t slots, const int* list, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int s = list[i];
    if (s >= 0 && s < slots) live[s] = 0;
}

}  // namespace

hipError_t launch_pool_copy(const PoolParams& p, const int* src, const int* dst, int64_t n, bool in_place,
                            hipStream_t stream)
{
    const dim3 grid((unsigned)(n * p.piece0[p.n]));
    if (grid.x == 0) return hipSuccess;
    if (!in_place) {
        hipLaunchKernelGGL((pool_copy_kernel<kMove>), grid, dim3(256), 0, stream, p, src, dst, (int)n);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((pool_copy_kernel<kStage>), grid, dim3(256), 0, stream, p, src, dst, (int)n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((pool_copy_kernel<kFinish>), grid, dim3(256), 0, stream, p, src, dst, (int)n);
    return hipGetLastError();
}

hipError_t launch_pool_fork(const PoolParams& p, const int* live, int* live_out, const int* parents, int* children,
                            int* list, int64_t n, hipStream_t stream)
{
    hipLaunchKernelGGL(pool_fork_plan, dim3(1), dim3(1024), 0, stream, live, live_out, p.dst_slots, parents, children, list, n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || n == 0 || p.piece0[p.n] == 0) return e;
    hipLaunchKernelGGL(pool_move_kernel, dim3((unsigned)(n * p.piece0[p.n])), dim3(256), 0, stream, p, parents, children,
                       (const int*)nullptr);
    return hipGetLastError();
}

hipError_t launch_pool_compact(const PoolParams& p, const int* live, int* live_out, int* new_slot, int* count, int* list,
                               hipStream_t stream)
{
    const int64_t slots = p.dst_slots;
    hipLaunchKernelGGL(pool_compact_plan, dim3(1), dim3(1024), 0, stream, live, live_out, slots, new_slot, count, list);
    const hipError_t e = hipGetLastError();
    const int64_t blocks = slots / 2 * p.piece0[p.n];
    if (e != hipSuccess || blocks == 0) return e;
    hipLaunchKernelGGL(pool_move_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p, list + 1, list + 1 + slots / 2, list);
    return hipGetLastError();
}

hipError_t launch_pool_free(int* live, int64_t slots, const int* list, int64_t n, hipStream_t stream)
{
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(pool_free_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, live, slots, list, n);
    return hipGetLastError();
}

}  // namespace m3
