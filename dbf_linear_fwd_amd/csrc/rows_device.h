// Rows in groups on the device (include/dbf.h, "Rows in groups").
#ifndef DBF_ROWS_DEVICE_H_
#define DBF_ROWS_DEVICE_H_

#include <hip/hip_runtime.h>

#include "dbf_internal.h"

namespace dbf {

// Places [lo, hi) of group e (e = count: of no group), whatever stands in offsets.
__device__ __forceinline__ void group_places(const int32_t *offsets, int count, int slots, int e, int &lo, int &hi) {
    const int first = offsets[e], next = offsets[min(e + 1, count)];  // (two loads at once)
    lo = min(max(first, 0), slots);
    hi = e < count ? min(max(next, lo), slots) : slots;
}

// The lanes of a wave see what each other wrote to LDS (whose accesses are in
// order for a wave: nothing is waited for).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Sum of v over the lanes up to this one: in rows of 16 lanes by row shifts,
// then the rows' last lanes into the rows behind (no LDS, as a shuffle takes).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // row_shr:1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);  // row_bcast:31 into rows 2 and 3
    return v;
}

// The largest of the lanes' values, none of them negative (their order is that of their bits).
__device__ __forceinline__ float wave_largest(float x) {
    int v = __builtin_bit_cast(int, x);
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(v, 63));
}

// Row tile `index` of the groups' tiles of `tile` places, group after group,
// those of no group (group = count) last: false past the last.  A wave finds
// it by itself, 64 groups at a time: two loads and a scan instead of a launch
// that writes a table.
__device__ __forceinline__ bool find_row_tile(const int32_t *offsets, int count, int slots, int tile, int index,
                                              RowTile &out) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 <= count; e0 += 64) {
        int lo = 0, hi = 0;
        if (e0 + lane <= count) group_places(offsets, count, slots, e0 + lane, lo, hi);
        const int tiles = (hi - lo + tile - 1) / tile;
        const int upto = before + wave_scan(tiles);
        const uint64_t past = __ballot(upto > index);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int first = __builtin_amdgcn_readlane(lo, at) +
                              (index - __builtin_amdgcn_readlane(upto - tiles, at)) * tile;
            out.group = e0 + at;
            out.first = first;
            out.rows = min(tile, __builtin_amdgcn_readlane(hi, at) - first);
            out.zero = 0;
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

}  // namespace dbf

#endif  // DBF_ROWS_DEVICE_H_
