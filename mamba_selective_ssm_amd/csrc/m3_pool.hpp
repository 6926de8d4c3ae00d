// Pools of state records: what the kernels and the ABI share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

constexpr int kPoolArrays = 8;
constexpr int kPoolPiece = 16384;   // bytes of a record that one workgroup moves

struct PoolParams {
    int n;                             // arrays of a record
    const char* src[kPoolArrays];
    char* dst[kPoolArrays];
    int64_t row[kPoolArrays];          // bytes of one slot in array i
    int unit[kPoolArrays];             // bytes per move, 16, 4, 2 or 1: divides row and the pieces' offsets
    int piece0[kPoolArrays + 1];       // first piece of array i in a record's pieces
    int64_t src_slots, dst_slots;
    char* ws;                          // staged records, ws_row bytes each (in-place copies)
    int64_t ws_row;
    int64_t ws_off[kPoolArrays];
};

// Pair i moves record src[i] to slot dst[i].
hipError_t launch_pool_copy(const PoolParams& p, const int* src, const int* dst, int64_t n, bool in_place,
                            hipStream_t stream);
hipError_t launch_pool_fork(const PoolParams& p, const int* live, int* live_out, const int* parents, int* children,
                            int* list, int64_t n, hipStream_t stream);
hipError_t launch_pool_compact(const PoolParams& p, const int* live, int* live_out, int* new_slot, int* count,
                               int* list, hipStream_t stream);
hipError_t launch_pool_free(int* live, int64_t slots, const int* list, int64_t n, hipStream_t stream);

}  // namespace m3
