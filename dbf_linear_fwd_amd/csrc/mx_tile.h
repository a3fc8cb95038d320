// What the tiled products of the block formats share: LDS loads and waits,
// the order of the tiles, and the way of a tile's sums to memory.
#ifndef DBF_MX_TILE_H_
#define DBF_MX_TILE_H_

#include <algorithm>
#include <atomic>
#include <cmath>

#include "mx_device.h"
#include "rows_device.h"

namespace dbf {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Operand words of a scaled matrix-core instruction (an e2m1 operand: a alone).
__device__ __forceinline__ i32x8 operand(u32v4 a, u32v4 b) {
    return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                 static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ void dma16(const void *g, char *l) {
    __builtin_amdgcn_global_load_lds(g, (lds_void *)(l), 16, 0, 0);
}
__device__ __forceinline__ void dma4(const void *g, char *l) {
    __builtin_amdgcn_global_load_lds(g, (lds_void *)(l), 4, 0, 0);
}

// Wait until at most N of this wave's loads are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    // vmcnt bits [3:0] and [15:14]; expcnt [6:4] and lgkmcnt [11:8] left at "no wait"
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// This wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }

// Nothing moves across in the compiler's schedule.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ void block_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int V>
using Const = std::integral_constant<int, V>;

// XCD-aware position of workgroup b among G: the workgroups of one XCD
// (b mod 8) take consecutive indexes, so that they share operands in its L2.
__device__ __forceinline__ int xcd_index(int b, int G) {
    constexpr int kXcds = 8;
    const int xcd = b % kXcds, slot = b / kXcds, q = G / kXcds, rem = G % kXcds;
    return xcd * q + min(xcd, rem) + slot;
}

// Tiles of an output and how workgroups go through them.
struct TileGrid {
    int nbm, nbn, nsplit;  // tile rows and columns, K parts
    int group;             // tile rows that consecutive workgroups go through first; of rows in groups: a
                           // round's workgroups (GroupedWork)
};

// Output tile of position `tile`: bands of `group` tile rows, column by
// column within a band, so that the tiles which run on one XCD at a time
// form a block that shares its rows of x and of the weight in that XCD's L2.
__device__ __forceinline__ void tile_at(const TileGrid &a, int tile, int &bm, int &bn) {
    const int band = tile / (a.group * a.nbn);
    const int rows = min(a.group, a.nbm - band * a.group);
    const int at = tile - band * a.group * a.nbn;
    bn = at / rows;
    bm = band * a.group + at - bn * rows;
}

// The rows of one tile of a product on rows in groups (MxRows).
struct RowPlaces {
    int first = 0;      // the tile's first place in the grouped order
    bool none = false;  // rows of no group
    // row of the input / of the result for row r of the tile (-1: not written)
    __device__ __forceinline__ int64_t in(const MxRows &a, int r) const {
        int64_t at = first + r;
        if (a.per > 0) at = a.order[at] / a.per;
        return at < 0 ? 0 : at < a.in_rows ? at : a.in_rows - 1;
    }
    __device__ __forceinline__ int64_t out(const MxRows &a, int r) const {
        const int64_t at = a.scatter ? a.order[first + r] : first + r;
        return at < a.slots ? at : -1;
    }
};

// The row tiles of a product, as a wave sees them (RowTile says their order).
struct RowTiles {
    int work = 0, total = 0;                  // of the groups; those of no group too
    bool few = false;                         // no tile is more than half full
    int large_all = 0, large, upto, small_upto, lo, hi;  // without a table: lane e has group e
};
template <int BM>
__device__ __forceinline__ RowTiles scan_rows(const MxRows &a) {
    RowTiles t;
    if (a.table) {
        const RowTile r = a.table[0];
        t.work = r.group;
        t.total = r.first;
        t.few = r.rows == 0;
        return t;
    }
    const int lane = threadIdx.x & 63;
    t.lo = t.hi = 0;
    if (lane < a.count) group_places(a.offsets, a.count, a.slots, lane, t.lo, t.hi);
    int lo, hi;
    group_places(a.offsets, a.count, a.slots, a.count, lo, hi);
    const int c = t.hi - t.lo, rest = c % BM;
    t.large = c / BM + (rest > BM / 2);
    t.upto = wave_scan(t.large);
    t.small_upto = wave_scan(rest > 0 && rest <= BM / 2);
    t.large_all = __builtin_amdgcn_readlane(t.upto, 63);
    t.few = t.large_all == 0;
    // (never more than an order's groups make: the grid and the parts' memory are for so many)
    const int most = static_cast<int>(row_tiles_bound(a.slots, a.count, BM));
    t.work = min(t.large_all + __builtin_amdgcn_readlane(t.small_upto, 63), most);
    t.total = __builtin_amdgcn_readfirstlane(min(t.work + (hi - lo + BM - 1) / BM, most));
    return t;
}

// The rows of row tile bm, and their group's weight in place of the first.
template <int BM>
__device__ __forceinline__ RowPlaces take_group(const MxRows &a, const RowTiles &t, int bm, MxWeight &w, int &M) {
    RowPlaces p;
    int e;
    if (a.table) {
        const RowTile r = a.table[1 + bm];
        e = r.group;
        p.first = r.first;
        M = r.rows;
    } else {
        int lo, hi, at;
        if (bm < t.large_all) {
            e = __builtin_ctzll(__ballot(t.upto > bm));
            lo = __builtin_amdgcn_readlane(t.lo, e);
            hi = __builtin_amdgcn_readlane(t.hi, e);
            at = bm - __builtin_amdgcn_readlane(t.upto - t.large, e);
        } else if (bm < t.work) {
            e = __builtin_ctzll(__ballot(t.small_upto > bm - t.large_all));
            lo = __builtin_amdgcn_readlane(t.lo, e);
            hi = __builtin_amdgcn_readlane(t.hi, e);
            at = (hi - lo) / BM;
        } else {
            e = a.count;
            group_places(a.offsets, a.count, a.slots, e, lo, hi);
            at = bm - t.work;
        }
        p.first = __builtin_amdgcn_readfirstlane(lo + at * BM);
        M = __builtin_amdgcn_readfirstlane(min(BM, hi - (lo + at * BM)));
    }
    p.none = e >= a.count;
    const size_t at = p.none ? 0 : e;
    w.codes += at * a.code_stride;
    w.scales += at * a.scale_stride;
    w.colmax += at * a.colmax_stride;
    return p;
}

// What workgroup b of a grouped product does.  The groups' tiles go over the
// CUs in rounds of `room` workgroups; those of the last round that would not
// fill it are cut into up to nsplit parts of K (4 steps at least).  An XCD
// (b % 8) keeps to its eighth of the columns where they divide, so that its
// part of the weights stays in its L2 for all row tiles, and every XCD has
// the same work; where groups have few rows, and every tile has a weight of its
// own, neighbouring workgroups take neighbouring columns (128 rows of 64 groups,
// 4096 x 1024: 26 instead of 28 us).  Tiles of no group come last.
struct GroupedWork {
    int bm = -1, bn = 0;             // bm < 0: nothing
    int split = 0, nsplit = 1;
    int cut = 0, at = 0;             // tiles that are cut, and the place of this one among them
};
__device__ __forceinline__ void place_tile(int p, int nbn, bool few, GroupedWork &w) {
    if (nbn % 8 == 0 && !few) {
        const int per = nbn / 8, q = p >> 3;
        w.bm = q / per;
        w.bn = (p & 7) * per + q - w.bm * per;
    } else {
        w.bm = p / nbn;
        w.bn = p - w.bm * nbn;
    }
}
// The tiles that are cut, from `head` on, and into how many parts.
__device__ __forceinline__ void cut_tiles(int tiles, int steps, int room, int most, int &head, int &parts) {
    head = tiles / room * room;
    const int cut = tiles - head;
    parts = cut > 0 ? min(min(room / cut, most), steps / 4) : 1;
    if (parts < 2) {
        parts = 1;
        head = tiles;
    }
}
__device__ __forceinline__ GroupedWork grouped_work(const RowTiles &t, int nbn, int steps, int room, int most, int b) {
    GroupedWork w;
    int head, parts;
    const int tiles = t.work * nbn;
    cut_tiles(tiles, steps, room, most, head, parts);
    w.cut = tiles - head;
    if (b < head) {
        place_tile(b, nbn, t.few, w);
    } else if (b < head + w.cut * parts) {
        w.split = (b - head) / w.cut;
        w.at = b - head - w.split * w.cut;
        w.nsplit = parts;
        place_tile(head + w.at, nbn, t.few, w);
    } else {
        const int i = b - (head + w.cut * parts);
        if (i < (t.total - t.work) * nbn) {
            w.bm = t.work + i / nbn;
            w.bn = i % nbn;
        }
    }
    return w;
}
// Workgroups of a grid for row tiles of BM, and tiles whose parts need memory.
inline int64_t grouped_grid(int64_t row_tiles, int nbn, int room) { return row_tiles * nbn + room; }

// Row tiles of `bm` places to reckon with where `count` groups share `slots`
// rows: the sizes are on the device, so they are taken to be spread as routers
// spread them, exponentially around their mean, whose tiles are geometric.
inline int64_t grouped_row_tiles(int slots, int count, int bm) {
    const int used = slots < count ? slots : count;
    return static_cast<int64_t>(used / (1.0 - std::exp(-static_cast<double>(bm) * used / slots)) + 0.5);
}

// Cost of a tile of a grouped product in microseconds: a workgroup with few
// others, start and step, and its share of a full CU.  K steps are cheaper and
// starts dearer than where one weight serves all workgroups: a tile has few
// rows of its own, and many starts overlap on a CU.
struct GroupedCost {
    float light0, light, full0, full;
    float time(int steps, float per_cu) const { return std::max(light0 + steps * light, per_cu * (full0 + steps * full)); }
};
// Estimated time of `tiles` tiles of bm x bn, `room` to a round (alone: one to
// a CU), with or without the last round's cut into up to `most` parts; a join
// costs its launch and the traffic of the parts.
inline float grouped_estimate(const GroupedCost &c, int64_t tiles, int steps, int room, bool alone, int most, int bm, int bn,
                              bool cut) {
    constexpr float kCus = 256.0f;
    const int64_t head = tiles / room * room, rest = tiles - head;
    const int parts = rest > 0 ? static_cast<int>(std::min<int64_t>({most, steps / 4, room / rest})) : 1;
    if (!cut || parts < 2) {
        const float per_cu = tiles / kCus;
        return c.time(steps, alone && per_cu < 8.0f ? std::ceil(per_cu) : per_cu) + (cut ? 3.0f : 0.0f);
    }
    return head / kCus * (c.full0 + steps * c.full) + c.time((steps + parts - 1) / parts, rest * parts / kCus) + 3.0f +
           static_cast<float>(rest * parts) * bm * bn * 8.0f * 2e-7f;
}

// A wave's results to y.  A 32 x 32 result has one row of y per lane, its
// columns 8 (v / 4) + 4 g + v % 4 in register v; each wave takes them through
// its own part of LDS (store_bytes at `mine`) into rows of 16-byte stores.  (Stored from the
// registers, two bytes a lane: 106 instead of 101 us, 256 x 256 tiles of
// 2048 x 14336, K 4096.)
template <typename C>
constexpr size_t store_bytes() { return 32 * (64 * C::NI + 16); }

// row_of(r): where row r < M of the results lies in y, -1: nowhere.
template <typename C, typename E, typename R>
__device__ __forceinline__ void store_tile(char *mine, const f32x16 (&acc)[C::MI][C::NI], void *out, int M,
                                           int n, int m0, int n0, int wave, int lane, R row_of) {
    const int wm = wave / C::WN, wn = wave % C::WN, l32 = lane & 31, g = lane >> 5;
    constexpr int Cols = 32 * C::NI, Pitch = Cols * 2 + 16;  // 16-bit values of a wave's row, bytes
    static_assert(store_bytes<C>() == 32 * Pitch, "");
    uint16_t *y = static_cast<uint16_t *>(out);
    const int c0 = n0 + wn * Cols;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
        const int r0 = m0 + (wm * C::MI + i) * 32;
#pragma unroll
        for (int f = 0; f < C::NI; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t p[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float lo = acc[i][f][4 * q + 2 * h], hi = acc[i][f][4 * q + 2 * h + 1];
                    p[h] = static_cast<uint32_t>(E::put(lo)) | static_cast<uint32_t>(E::put(hi)) << 16;
                }
                *reinterpret_cast<u32v2 *>(mine + l32 * Pitch + (f * 32 + 8 * q + 4 * g) * 2) = u32v2{p[0], p[1]};
            }
        // (rows of any alignment: the memory takes unaligned stores; two bytes
        // at a time, 5376 rows of ten groups, 5518 x 64, 98 us)
        typedef u32v4 u32v4_any __attribute__((aligned(2)));
        constexpr int Per = Cols / 8, Rows = 64 / Per;  // lanes per row, rows per store
        const int c = lane % Per * 8;
#pragma unroll
        for (int j = 0; j < 32; j += Rows) {
            const int r = j + lane / Per;
            const u32v4 v = *reinterpret_cast<const u32v4 *>(mine + r * Pitch + c * 2);
            if (r0 + r < M && c0 + c < n) {
                const int64_t at = row_of(r0 + r);
                if (at < 0) continue;
                uint16_t *dst = y + static_cast<size_t>(at) * n + c0 + c;
                if (c0 + c + 8 <= n) {
                    *reinterpret_cast<u32v4_any *>(dst) = v;
                } else {
                    for (int k = 0; k < n - c0 - c; ++k)
                        dst[k] = *reinterpret_cast<const uint16_t *>(mine + r * Pitch + (c + k) * 2);
                }
            }
        }
    }
}

template <typename C, typename E>
__device__ __forceinline__ void store_tile(char *mine, const f32x16 (&acc)[C::MI][C::NI], void *out, int M,
                                           int n, int m0, int n0, int wave, int lane) {
    store_tile<C, E>(mine, acc, out, M, n, m0, n0, wave, lane, [](int r) { return static_cast<int64_t>(r); });
}

// The sums of a K part of a tile as they are (a wave's 1024 floats per 32 x 32
// result, 16 bytes a lane), and the parts of a tile added in order.
template <typename C>
__device__ __forceinline__ float *part_at(float *part, int split, int tiles, int tile, int wave, int lane) {
    return part + ((static_cast<size_t>(split) * tiles + tile) * C::Waves + wave) * (C::MI * C::NI * 1024) + lane * 4;
}

template <typename C>
__device__ __forceinline__ void store_part(float *p, const f32x16 (&acc)[C::MI][C::NI]) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int f = 0; f < C::NI; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4 *>(p + ((i * C::NI + f) * 4 + q) * 256) =
                    f32x4{acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3]};
}

template <typename C>
__device__ __forceinline__ void add_parts(const float *p, size_t plane, int nsplit, f32x16 (&acc)[C::MI][C::NI]) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int f = 0; f < C::NI; ++f)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][f][v] = 0.0f;
#pragma unroll C::MI * C::NI == 1 ? 4 : 1
    for (int s = 0; s < nsplit; ++s, p += plane)
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
            for (int f = 0; f < C::NI; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(p + ((i * C::NI + f) * 4 + q) * 256);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][f][4 * q + e] += v[e];
                }
}

// More than 64 KiB of LDS has to be asked for, once per kernel and device.
template <typename K>
void allow_lds(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    (void)hipGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return;
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes));
    done.fetch_or(bit, std::memory_order_relaxed);
}

}  // namespace
}  // namespace dbf

#endif  // DBF_MX_TILE_H_
