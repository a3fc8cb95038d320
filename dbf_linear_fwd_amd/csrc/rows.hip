// Rows in groups: the stable sort of rows by group, and the table of a grouped
// product's row tiles.
//
// The sort counts and places (keys are few: groups plus one for no group).  A
// wave goes through consecutive rows, 64 at a time; the lanes of one key find
// each other by a ballot per bit of the key, so a row's place is its key's
// next place plus the lanes of its key below it, and no atomic is needed:
// the order is that of the rows.  Counts of each wave stand in LDS and are
// summed over the keys before and the waves before.
//
// Latency is all it costs.  Up to 4096 rows are one workgroup and one launch;
// more are cut into workgroups of 1024, 4096 or 16384 rows, one launch that
// counts and one that places, where every workgroup adds up the counts of the
// others (of more than kDirectParts, a launch between does).  Graph replays, 64
// groups: 128 rows 4.4 us (16 steps of 64 rows unrolled, most of them skipped:
// 6.2), 2048 rows 5.9, 4096 8.0, 16384 8.9 (in one workgroup 22), 65536 10.9
// (in workgroups of 4096 rows 14.3), 262144 16.4 (of 16384 36), 2^20 39.

#include <algorithm>
#include <atomic>

#include "mx_tile.h"
#include "rows_device.h"

namespace dbf {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int block_rows(int steps) { return kThreads * steps; }  // steps of 64 rows per wave
constexpr int kMaxSteps = 16;
constexpr int kDirectParts = 64;
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
    const int incl = wave_scan(v);
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
    int32_t *counts;  // [workgroups][count + 1]: of each workgroup's keys; scanned: their first places
    int parts, scanned;
};

enum class Sort { Whole, Count, Place };

// Whole: all rows in one workgroup.  Count: the counts of a workgroup's rows
// to memory.  Place: its rows to their places.
template <typename I, Sort S, int Steps>
__global__ __launch_bounds__(kThreads) void sort_kernel(const SortArgs a) {
    extern __shared__ int hist[];  // [kWaves][keys]
    __shared__ int tmp[kWaves];
    const int keys = a.count + 1;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const I *index = static_cast<const I *>(a.index);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * block_rows(Steps);
    const int here = static_cast<int>(a.rows - first < block_rows(Steps) ? a.rows - first : block_rows(Steps));
    const int steps = ((here + 63) / 64 + kWaves - 1) / kWaves;  // per wave
    const int row0 = wave * steps * 64 + lane;

    for (int i = threadIdx.x; i < kWaves * keys; i += kThreads) hist[i] = 0;
    int key[Steps];
#pragma unroll
    for (int s = 0; s < Steps; ++s) {
        const int r = row0 + s * 64;
        if (s < steps && r < here) key[s] = key_of(index, first + r, a.count);
    }
    __syncthreads();
    int *mine = hist + wave * keys;
#pragma unroll
    for (int s = 0; s < Steps; ++s)
        if (s < steps) {
            const bool on = row0 + s * 64 < here;
            const uint64_t same = same_key(on ? key[s] : 0, a.bits, __ballot(on));
            if (on && (same & ((1ull << lane) - 1)) == 0) mine[key[s]] += __popcll(same);
            wave_fence();
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
            int start = 0, all = sum;  // of the workgroups before, and of all
            if constexpr (S == Sort::Place) {
                const int32_t *c = a.counts + k;
                if (a.scanned) {
                    if (k < keys) start = c[static_cast<size_t>(blockIdx.x) * keys];
                } else {
                    all = 0;
                    if (k < keys) {
#pragma unroll 8
                        for (int p = 0; p < a.parts; ++p) {
                            const int n = c[p * keys];
                            if (p < static_cast<int>(blockIdx.x)) start += n;
                            all += n;
                        }
                    }
                }
            }
            if (S == Sort::Whole || !a.scanned) {
                int total;
                const int at = before + block_scan(all, tmp, total);
                before += total;
                if (k < keys && blockIdx.x == 0) a.offsets[k] = at;
                start += at;
            }
            if (k < keys)
                for (int w = 0; w < kWaves; ++w) hist[w * keys + k] += start;
        }
    }
    if constexpr (S == Sort::Count) return;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < Steps; ++s)
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
            wave_fence();
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

// The row tiles of a grouped product, in the order that RowTile says.
__global__ __launch_bounds__(kThreads) void row_tiles_kernel(const int32_t *offsets, int count, int slots, int tile,
                                                             RowTile *table, int bound) {
    __shared__ int large_at[kMaxGroups + 1], small_at[kMaxGroups + 1], low[kMaxGroups + 1], high[kMaxGroups + 1];
    __shared__ int tmp[kWaves];
    int larges = 0, smalls = 0;
    for (int e0 = 0; e0 <= count; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int lo = 0, hi = 0;
        if (e <= count) group_places(offsets, count, slots, e, lo, hi);
        const int c = e < count ? hi - lo : 0, rest = c % tile;
        int total;
        const int l = larges + block_scan(c / tile + (rest > tile / 2), tmp, total);
        larges += total;
        const int s = smalls + block_scan(rest > 0 && rest <= tile / 2, tmp, total);
        smalls += total;
        if (e <= count) {
            large_at[e] = l;
            small_at[e] = s;
            low[e] = lo;
            high[e] = hi;
        }
    }
    __syncthreads();
    const int none_lo = low[count], nones = (high[count] - none_lo + tile - 1) / tile;
    const int work = min(larges + smalls, bound), all = min(work + nones, bound);
    if (threadIdx.x == 0) table[0] = RowTile{work, all, larges, 0};
    for (int t = threadIdx.x; t < all; t += kThreads) {
        RowTile r{count, none_lo + (t - work) * tile, 0, 0};
        if (t < work) {
            const bool large = t < larges;
            const int *at = large ? large_at : small_at, i = large ? t : t - larges;
            int e = 0;  // the last group that starts at or before i
            for (int step = 1024; step > 0; step >>= 1)
                if (e + step < count && at[e + step] <= i) e += step;
            r.group = e;
            r.first = low[e] + (large ? i - at[e] : (high[e] - low[e]) / tile) * tile;
        }
        r.rows = min(tile, high[r.group] - r.first);
        table[1 + t] = r;
    }
}

// Steps of a wave: one workgroup up to 4096 rows, then as many workgroups as add up each other's counts.
int sort_steps(int64_t rows) {
    for (int steps : {1, 2, 4})
        if (rows <= block_rows(steps)) return steps;
    for (int steps : {1, 4})
        if (rows <= static_cast<int64_t>(kDirectParts) * block_rows(steps)) return steps;
    return kMaxSteps;
}
int sort_parts(int64_t rows) {
    const int64_t per = block_rows(sort_steps(rows));
    return static_cast<int>(rows <= per ? 1 : (rows + per - 1) / per);
}
size_t sort_bytes(int64_t rows, int count) {
    const int parts = sort_parts(rows);
    return parts == 1 ? 0 : static_cast<size_t>(parts) * (count + 1) * sizeof(int32_t);
}

template <typename I, int Steps>
void launch_sort(SortArgs &a, hipStream_t s) {
    const size_t lds = sizeof(int) * kWaves * (a.count + 1);
    auto go = [&](auto kernel, std::atomic<uint64_t> &asked) {
        if (lds > 60 * 1024) allow_lds(kernel, sizeof(int) * kWaves * (kMaxGroups + 1), asked);
        launch_kernel(kernel, dim3(a.parts), dim3(kThreads), lds, s, a);
    };
    if (a.parts == 1) {
        if constexpr (Steps <= 4) {
            static std::atomic<uint64_t> whole{0};
            go(sort_kernel<I, Sort::Whole, Steps>, whole);
        }
        return;
    }
    if constexpr (Steps != 2) {
        static std::atomic<uint64_t> counting{0}, placing{0};
        go(sort_kernel<I, Sort::Count, Steps>, counting);
        if (a.scanned)
            launch_kernel(sort_scan_kernel, dim3(1), dim3(kThreads), 0, s, a.counts, a.parts, a.count + 1, a.offsets);
        go(sort_kernel<I, Sort::Place, Steps>, placing);
    }
}

template <typename I>
int launch_sort(SortArgs &a, hipStream_t s) {
    a.parts = sort_parts(a.rows);
    a.scanned = a.parts > kDirectParts;
    switch (sort_steps(a.rows)) {
        case 1: launch_sort<I, 1>(a, s); break;
        case 2: launch_sort<I, 2>(a, s); break;
        case 4: launch_sort<I, 4>(a, s); break;
        default: launch_sort<I, kMaxSteps>(a, s); break;
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
    SortArgs a{index, rows, count, 0, order, offsets, static_cast<int32_t *>(workspace), 1, 0};
    while ((1 << a.bits) < count + 1) ++a.bits;
    const int e = index_bits == 32 ? launch_sort<int32_t>(a, stream) : launch_sort<int64_t>(a, stream);
    return e == 0 ? DBF_OK : DBF_ERR_HIP;
}
