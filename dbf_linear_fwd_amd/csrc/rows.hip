// Rows in groups: the stable sort of rows by group, and the table of a grouped
// product's row tiles.
//
// The sort counts and places (keys are few: groups plus one for no group).  A
// wave goes through consecutive rows, 64 at a time; the lanes of one key find
// each other by a ballot per bit of the key, so a row's place is its key's
// next place plus the lanes of its key below it, and no atomic is needed:
// the order is that of the rows.  Counts of each wave stand in LDS and are
// summed over the keys before and the waves before.  Up to kBlockRows rows
// are one workgroup and one launch; more are one workgroup each, with a
// launch that adds up their counts between the counting and the placing.

#include <algorithm>
#include <atomic>

#include "mx_tile.h"
#include "rows_device.h"

namespace dbf {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kSteps = 16;                            // of 64 rows, per wave
constexpr int kBlockRows = kWaves * kSteps * 64;      // 16384
constexpr int kMaxGroups = 1024;
constexpr int64_t kMaxRows = int64_t(1) << 24;

template <typename I>
__device__ __forceinline__ int key_of(const I *index, int64_t row, int count) {
    const I v = index[row];
    return v >= 0 && v < static_cast<I>(count) ? static_cast<int>(v) : count;
}

// Lanes (of those in `on`) that hold the same key.
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t on) {
    uint64_t m = on;
    for (int b = 0; b < bits; ++b) {
        const bool bit = key >> b & 1;
        const uint64_t s = __ballot(bit);
        m &= bit ? s : ~s;
    }
    return m;
}

// Exclusive sum over the workgroup's threads; total is everyone's.
__device__ __forceinline__ int block_scan(int v, int *tmp, int &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int incl = wave_scan(v, lane);
    if (lane == 63) tmp[wave] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += tmp[w];
        total += tmp[w];
    }
    __syncthreads();
    return before + incl - v;
}

struct SortArgs {
    const void *index;
    int64_t rows;
    int count, bits;
    int32_t *order, *offsets;
    int32_t *counts;  // [workgroups][count + 1]: of each workgroup's keys, then their first places
};

enum class Sort { Whole, Count, Place };

// Whole: all rows in one workgroup.  Count: the counts of a workgroup's rows
// to memory.  Place: its rows to their places, from the first places there.
template <typename I, Sort S>
__global__ __launch_bounds__(kThreads) void sort_kernel(const SortArgs a) {
    extern __shared__ int hist[];  // [kWaves][keys]
    __shared__ int tmp[kWaves];
    const int keys = a.count + 1;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const I *index = static_cast<const I *>(a.index);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kBlockRows;
    const int here = static_cast<int>(a.rows - first < kBlockRows ? a.rows - first : kBlockRows);
    const int steps = ((here + 63) / 64 + kWaves - 1) / kWaves;  // per wave
    const int row0 = wave * steps * 64 + lane;

    for (int i = threadIdx.x; i < kWaves * keys; i += kThreads) hist[i] = 0;
    int key[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int r = row0 + s * 64;
        if (s < steps && r < here) key[s] = key_of(index, first + r, a.count);
    }
    __syncthreads();
    int *mine = hist + wave * keys;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
        if (s < steps) {
            const bool on = row0 + s * 64 < here;
            const uint64_t same = same_key(on ? key[s] : 0, a.bits, __ballot(on));
            if (on && (same & ((1ull << lane) - 1)) == 0) mine[key[s]] += __popcll(same);
        }
    __syncthreads();
    // the waves' counts of a key become their places behind the waves before
    for (int k0 = 0, before = 0; k0 < keys; k0 += kThreads) {
        const int k = k0 + threadIdx.x;
        int sum = 0;
        if (k < keys)
            for (int w = 0; w < kWaves; ++w) {
                const int c = hist[w * keys + k];
                hist[w * keys + k] = sum;
                sum += c;
            }
        if constexpr (S == Sort::Count) {
            if (k < keys) a.counts[static_cast<size_t>(blockIdx.x) * keys + k] = sum;
        } else {
            int start;
            if constexpr (S == Sort::Whole) {
                int total;
                start = before + block_scan(sum, tmp, total);
                before += total;
                if (k < keys) a.offsets[k] = start;
            } else {
                start = k < keys ? a.counts[static_cast<size_t>(blockIdx.x) * keys + k] : 0;
            }
            if (k < keys)
                for (int w = 0; w < kWaves; ++w) hist[w * keys + k] += start;
        }
    }
    if constexpr (S == Sort::Count) return;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
        if (s < steps) {
            const bool on = row0 + s * 64 < here;
            const uint64_t same = same_key(on ? key[s] : 0, a.bits, __ballot(on));
            const uint64_t below = same & ((1ull << lane) - 1);
            if (on) {
                const int at = mine[key[s]] + __popcll(below);
                a.order[at] = static_cast<int32_t>(first + row0 + s * 64);
                // (a wave's LDS accesses are in order: every lane has read its place)
                if (below == 0) mine[key[s]] = at + __popcll(same);
            }
        }
}

// Counts of the workgroups into first places.
__global__ __launch_bounds__(kThreads) void sort_scan_kernel(int32_t *counts, int parts, int keys, int32_t *offsets) {
    __shared__ int tmp[kWaves];
    for (int k0 = 0, before = 0; k0 < keys; k0 += kThreads) {
        const int k = k0 + threadIdx.x;
        int sum = 0;
        if (k < keys)
            for (int p = 0; p < parts; ++p) sum += counts[static_cast<size_t>(p) * keys + k];
        int total;
        int at = before + block_scan(sum, tmp, total);
        before += total;
        if (k < keys) {
            offsets[k] = at;
            for (int p = 0; p < parts; ++p) {
                int32_t *c = counts + static_cast<size_t>(p) * keys + k;
                const int n = *c;
                *c = at;
                at += n;
            }
        }
    }
}

// The row tiles of a grouped product, those of no group last.
__global__ __launch_bounds__(kThreads) void row_tiles_kernel(const int32_t *offsets, int count, int slots, int tile,
                                                             RowTile *table, int bound) {
    __shared__ int start[kMaxGroups + 1], low[kMaxGroups + 1], high[kMaxGroups + 1];
    __shared__ int tmp[kWaves];
    int before = 0;
    for (int e0 = 0; e0 <= count; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int lo = 0, hi = 0;
        if (e <= count) group_places(offsets, count, slots, e, lo, hi);
        const int tiles = (hi - lo + tile - 1) / tile;
        int total;
        const int at = before + block_scan(tiles, tmp, total);
        before += total;
        if (e <= count) {
            start[e] = at;
            low[e] = lo;
            high[e] = hi;
        }
    }
    __syncthreads();
    const int all = min(before, bound);
    if (threadIdx.x == 0) table[0] = RowTile{all, 0, 0, 0};
    for (int t = threadIdx.x; t < all; t += kThreads) {
        int e = 0;  // the last group that starts at or before t
        for (int step = 1024; step > 0; step >>= 1)
            if (e + step <= count && start[e + step] <= t) e += step;
        const int first = low[e] + (t - start[e]) * tile;
        table[1 + t] = RowTile{e, first, min(tile, high[e] - first), 0};
    }
}

size_t sort_bytes(int64_t rows, int count) {
    return rows <= kBlockRows ? 0 : static_cast<size_t>((rows + kBlockRows - 1) / kBlockRows) * (count + 1) * sizeof(int32_t);
}

template <typename I>
int launch_sort(SortArgs &a, hipStream_t s) {
    static std::atomic<uint64_t> whole{0}, counting{0}, placing{0};
    const size_t lds = sizeof(int) * kWaves * (a.count + 1);
    auto go = [&](auto kernel, std::atomic<uint64_t> &asked, uint32_t grid) {
        allow_lds(kernel, sizeof(int) * kWaves * (kMaxGroups + 1), asked);
        launch_kernel(kernel, dim3(grid), dim3(kThreads), lds, s, a);
    };
    if (a.rows <= kBlockRows) {
        go(sort_kernel<I, Sort::Whole>, whole, 1);
    } else {
        const uint32_t parts = static_cast<uint32_t>((a.rows + kBlockRows - 1) / kBlockRows);
        go(sort_kernel<I, Sort::Count>, counting, parts);
        launch_kernel(sort_scan_kernel, dim3(1), dim3(kThreads), 0, s, a.counts, static_cast<int>(parts), a.count + 1,
                      a.offsets);
        go(sort_kernel<I, Sort::Place>, placing, parts);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_row_tiles(const int32_t *offsets, int count, int slots, int tile, RowTile *table, int64_t bound,
                     void *stream) {
    launch_kernel(row_tiles_kernel, dim3(1), dim3(kThreads), 0, static_cast<hipStream_t>(stream), offsets, count, slots,
                  tile, table, static_cast<int>(bound));
    return static_cast<int>(hipGetLastError());
}

}  // namespace dbf

extern "C" size_t dbf_group_rows_workspace(int32_t rows, int32_t count) {
    if (rows < 1 || count < 1 || count > dbf::kMaxGroups || rows > dbf::kMaxRows) return 0;
    return dbf::sort_bytes(rows, count);
}

extern "C" dbf_status_t dbf_group_rows(const void *index, int32_t index_bits, int32_t rows, int32_t count,
                                       int32_t *order, int32_t *offsets, void *workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    using namespace dbf;
    if (rows < 0 || count < 1 || (index_bits != 32 && index_bits != 64)) return DBF_ERR_INVALID_ARG;
    if (count > kMaxGroups || rows > kMaxRows) return DBF_ERR_SHAPE;
    auto aligned = [](const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (!aligned(offsets, 4)) return DBF_ERR_INVALID_ARG;
    if (rows > 0 && (!aligned(index, index_bits / 8) || !aligned(order, 4))) return DBF_ERR_INVALID_ARG;
    const size_t need = sort_bytes(rows, count);
    if (need > 0 && (!aligned(workspace, 4) || workspace_bytes < need)) return DBF_ERR_INVALID_ARG;
    SortArgs a{index, rows, count, 0, order, offsets, static_cast<int32_t *>(workspace)};
    while ((1 << a.bits) < count + 1) ++a.bits;
    const int e = index_bits == 32 ? launch_sort<int32_t>(a, stream) : launch_sort<int64_t>(a, stream);
    return e == 0 ? DBF_OK : DBF_ERR_HIP;
}
