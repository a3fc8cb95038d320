// What the tiled products of the block formats share: LDS loads and waits,
// the order of the tiles, and the way of a tile's sums to memory.
#ifndef DBF_MX_TILE_H_
#define DBF_MX_TILE_H_

#include <atomic>

#include "mx_device.h"

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
    int group;             // tile rows that consecutive workgroups go through first
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

// A wave's results to y.  A 32 x 32 result has one row of y per lane, its
// columns 8 (v / 4) + 4 g + v % 4 in register v; each wave takes them through
// its own part of LDS (store_bytes at `mine`) into rows of 16-byte stores.  (Stored from the
// registers, two bytes a lane: 106 instead of 101 us, 256 x 256 tiles of
// 2048 x 14336, K 4096.)
template <typename C>
constexpr size_t store_bytes() { return 32 * (64 * C::NI + 16); }

template <typename C, typename E>
__device__ __forceinline__ void store_tile(char *mine, const f32x16 (&acc)[C::MI][C::NI], void *out, int M,
                                           int n, int m0, int n0, int wave, int lane) {
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
        if (n % 8 == 0) {
            constexpr int Per = Cols / 8, Rows = 64 / Per;  // lanes per row, rows per store
            const int c = lane % Per * 8;
#pragma unroll
            for (int j = 0; j < 32; j += Rows) {
                const int r = j + lane / Per;
                const u32v4 v = *reinterpret_cast<const u32v4 *>(mine + r * Pitch + c * 2);
                if (r0 + r < M && c0 + c < n)
                    *reinterpret_cast<u32v4 *>(y + static_cast<size_t>(r0 + r) * n + c0 + c) = v;
            }
        } else {
            for (int j = lane; j < 32 * Cols; j += 64) {
                const int r = j / Cols, c = j % Cols;
                if (r0 + r < M && c0 + c < n)
                    y[static_cast<size_t>(r0 + r) * n + c0 + c] =
                        *reinterpret_cast<const uint16_t *>(mine + r * Pitch + c * 2);
            }
        }
    }
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
