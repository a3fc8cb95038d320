// Low-rank adapters of rows in groups, and their gradients (include/dbf.h).
//
//   t = x A_aᵀ          y  = base + s_a t B_aᵀ
//   u = s_a dy B_a      dx' = dx + u A_a     dA_a = Σ u xᵀ    dB_a = s_a Σ dy tᵀ
//
// Kernels on the 16x16x32 16-bit matrix-core instructions, operands from
// memory straight into registers:
//   shrink  rows x K -> rows x rank (t, u): K cut between the waves of a
//           workgroup and into parts, whose fp32 sums go to memory;
//   expand  rows x rank -> rows x columns (y, dx'): a workgroup adds the parts
//           of its row tile's t into LDS and goes through its columns;
//   outer   the sums over a group's rows (dA, dB): the rows of a group in
//           chunks, joined in order by outer_join where a group has several.
// A product needs no more than 2 rank operations per element of x, dy or y, so
// the rows' memory traffic is the bound, and with few rows the launches.
// Measured (kernel trace; bytes as they have to be moved): 8192 rows, 4096 +
// 4096, rank 16, bf16: shrink 14 us (67 MB, 4.7 TB/s), expand 28 (134 MB, 4.7),
// outer 29 (134 MB, 4.7) and its join 5; 2048 rows, m 4096, n 14336, rank 64:
// shrink 13 us, expand 37 (117 MB, 3.1 TB/s); 16 rows of 32 adapters, 4096 x
// 4096, rank 16, f16: 3.4 and 5.3 us, 8.2 for both in a graph (in one launch,
// every workgroup with all of its t: 9.1).
//
// Of an instruction a lane (c = lane % 16, g = lane / 16) supplies row c of each
// operand, eight values of K from 8 g on, and gets results 4 g .. 4 g + 3 of
// the first operand for row c of the second.  An operand that has K contiguous
// in memory is one 16-byte load; one with K along the rows (B in u, A in dx',
// x and dy in the gradients) is loaded as eight rows of neighbouring columns
// and its halves are picked by byte permutes, four per operand.
//
// t and u stay fp32 in memory and become 16-bit operands in parts: f16 two
// parts of t 2^k, k from the largest of the row (of a wave's rows so far in
// the gradients), 2^-23 of each value or 2^-39 of that largest; bf16 two parts
// (2^-17) where a 16-bit result follows, three (24 bits) for the fp32 gradients.

#include <algorithm>

#include "mx_tile.h"
#include "rows_device.h"

namespace dbf {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMaxRank = 128, kMaxGroups = 1024;
constexpr int kMaxParts = 16;

template <typename E>
__device__ __forceinline__ f32x4 mma(u32v4 a, u32v4 b, f32x4 acc) {
    if constexpr (E::code == DBF_TYPE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
}

// 16-byte and shorter accesses at any element (the memory takes them unaligned).
typedef u32v4 u32v4_any __attribute__((aligned(2)));
typedef u32v2 u32v2_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// N consecutive 16-bit elements from p into words, the first `valid` of them
// (VEC: all or none), zeros for the rest.
template <int N, bool VEC>
__device__ __forceinline__ void load_n(const uint16_t *p, int valid, uint32_t (&w)[(N + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (N + 1) / 2; ++i) w[i] = 0;
    if (valid <= 0) return;
    if (VEC || valid >= N) {
        if constexpr (N == 1) w[0] = *p;
        else if constexpr (N == 2) w[0] = *reinterpret_cast<const u32_any *>(p);
        else if constexpr (N == 4) {
            const u32v2 v = *reinterpret_cast<const u32v2_any *>(p);
            w[0] = v[0];
            w[1] = v[1];
        } else {
            const u32v4 v = *reinterpret_cast<const u32v4_any *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < valid) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
}

template <bool VEC>
__device__ __forceinline__ u32v4 load_row8(const uint16_t *p, int valid) {
    uint32_t w[4];
    load_n<8, VEC>(p, valid, w);
    return u32v4{w[0], w[1], w[2], w[3]};
}

// Element i of eight rows of N: the operand whose K runs along the rows.
template <int N>
__device__ __forceinline__ u32v4 pick_column(const uint32_t (&q)[8][(N + 1) / 2], int i) {
    const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;  // the high or the low halves of (second, first)
    u32v4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __builtin_amdgcn_perm(q[2 * k + 1][i >> 1], q[2 * k][i >> 1], sel);
    return r;
}

// Two neighbouring values of part P (0, 1, 2) of v: rounded to 16 bits, the
// rest of that rounded, the rest of that.  EDGE: a finite v above bf16's largest
// value has that one for its first part, and a rest that the second holds.
template <typename E, bool EDGE>
__device__ __forceinline__ uint16_t part_of(float v, int part) {
    uint16_t h = E::put(v);
    if constexpr (EDGE && E::code == DBF_TYPE_BF16)
        if ((h & 0x7fff) == 0x7f80 && __builtin_isfinite(v)) --h;
    for (int p = 0; p < part; ++p) {
        const float top = E::get(h);
        v = __builtin_isfinite(top) ? v - top : 0.0f;
        h = E::put(v);
    }
    return h;
}
template <typename E, bool EDGE>
__device__ __forceinline__ u32v4 pack_part(const float (&v)[8], int part) {
    u32v4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = static_cast<uint32_t>(part_of<E, EDGE>(v[2 * i], part)) | static_cast<uint32_t>(part_of<E, EDGE>(v[2 * i + 1], part)) << 16;
    return r;
}

// Infinities.  A part of t or u that is 0, or of the other sign than the first,
// makes NaN of an infinite factor.  Where a sum is not finite, the same sum over
// the signs of its factors (0, 1, -1, infinities and NaN as they are; one
// product, no parts) says what the formula has there: if that is not finite,
// it is the result.  8192 rows, 4096 + 4096, rank 16, bf16, gradients: 69 us, with
// one infinity in x and in dy 166, with nothing else 243.
template <typename E>
constexpr uint32_t kInf16 = E::code == DBF_TYPE_BF16 ? 0x7f80u : 0x7c00u;
template <typename E>
constexpr uint32_t kOne16 = E::code == DBF_TYPE_BF16 ? 0x3f80u : 0x3c00u;
template <typename E>
__device__ __forceinline__ uint32_t sign16(uint32_t v) {
    const uint32_t size = v & 0x7fffu;
    return size == 0 ? 0u : size >= kInf16<E> ? v : (v & 0x8000u) | kOne16<E>;
}
template <typename E>
__device__ __forceinline__ uint32_t sign16(float v) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, v), size = bits & 0x7fffffffu;
    const uint32_t code = size == 0 ? 0u : size < 0x7f800000u ? kOne16<E> : size == 0x7f800000u ? kInf16<E> : 0x7fffu;
    return code | (bits >> 16 & 0x8000u);
}
template <typename E>
__device__ __forceinline__ u32v4 signs(u32v4 w) {
    u32v4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = sign16<E>(w[i] & 0xffffu) | sign16<E>(w[i] >> 16) << 16;
    return r;
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

// The power of two that brings `top` (a largest magnitude) to [2^14, 2^15).
__device__ __forceinline__ int f16_shift(float top) {
    int ex = 0;
    (void)frexpf(top, &ex);
    return top > 0.0f ? 15 - ex : 0;
}
constexpr int kNoShift = 200;  // (more than any value's)
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;  // (a NaN: 0)
}

// ---------------------------------------------------------------------------

struct ShrinkArgs {
    const uint16_t *x, *w;      // rows x K; count x rank x K, or (LEAD) count x K x rank
    const int32_t *order, *offsets;
    int rows, K, rank, count, parts;
    float *out;                 // [parts][rows][16 RT], by place
};

// MT tiles of 16 rows, ranks c RT + i (i < RT) in lane c's operand i.  Of large
// launches two thirds of the time are the first loads' way: a workgroup's few
// steps (2048 rows, K 4096, rank 64: four of 32 columns per wave) are little
// more than one wait.  More steps in flight change nothing there, twice the
// workgroups cost 4 us in both products.
template <typename E, bool LEAD, int MT, int RT, bool VEC>
__global__ __launch_bounds__(kThreads) void shrink_kernel(const ShrinkArgs a) {
    constexpr int RP = 16 * RT, Rows = 16 * MT, Pitch = RP + 4;
    __shared__ __attribute__((aligned(16))) float red[kWaves][16][Pitch];
    const int tile = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    RowTile rt;
    if (!find_row_tile(a.offsets, a.count, a.rows, Rows, tile, rt) || rt.group >= a.count) return;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int steps = (a.K + 31) / 32, pw = part * kWaves + wave, all = a.parts * kWaves;
    const int k0 = static_cast<int>(static_cast<int64_t>(pw) * steps / all);
    const int k1 = static_cast<int>(static_cast<int64_t>(pw + 1) * steps / all);
    const uint16_t *xr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = min(max(a.order[rt.first + min(16 * i + c, rt.rows - 1)], 0), a.rows - 1);
        xr[i] = a.x + static_cast<size_t>(row) * a.K + 8 * g;
    }
    const uint16_t *w = a.w + static_cast<size_t>(rt.group) * a.rank * a.K;
    f32x4 acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // U steps' operands are on their way at a time
    constexpr int U = MT + RT <= 3 ? 4 : MT + RT <= 6 ? 2 : 1;
    // XV: every lane has all of its eight columns or none; WV: its RT ranks
    auto turn = [&](int s0, auto xv, auto wv) {
        constexpr bool XV = decltype(xv)::value, WV = decltype(wv)::value;
        u32v4 xf[U][MT], wf[U][RT];
        uint32_t q[U][8][(RT + 1) / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = 32 * (s0 + u), left = s0 + u < k1 ? a.K - k - 8 * g : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[u][i] = load_row8<XV>(xr[i] + k, left);
            if constexpr (LEAD) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    load_n<RT, WV>(w + static_cast<size_t>(k + 8 * g + j) * a.rank + c * RT, j < left ? a.rank - c * RT : 0, q[u][j]);
            } else {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int j = c * RT + i;
                    wf[u][i] = load_row8<XV>(w + static_cast<size_t>(j) * a.K + k + 8 * g, j < a.rank ? left : 0);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (LEAD) {
#pragma unroll
                for (int i = 0; i < RT; ++i) wf[u][i] = pick_column<RT>(q[u], i);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[i][j] = mma<E>(wf[u][j], xf[u][i], acc[i][j]);
        }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    for (int s0 = k0; s0 < k1; s0 += U) {
        if (VEC) {
            turn(s0, Yes{}, Yes{});
        } else {
            // (only the last columns of an odd width are looked at one by one: 1491
            // rows, K 247, rank 128, 7 instead of 11 us)
            const bool full = 32 * (s0 + U) <= a.K, ranks = !LEAD || a.rank % RT == 0;
            if (full && ranks) turn(s0, Yes{}, Yes{});
            else if (ranks) turn(s0, No{}, Yes{});
            else turn(s0, No{}, No{});
        }
    }
    // lane (c, g): ranks (4 g + v) RT + i of row c; 16 rows at a time
    float *out = a.out + (static_cast<size_t>(part) * a.rows + rt.first) * RP;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if (16 * i >= rt.rows) break;
        if (i > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[wave][c][(4 * g + v) * RT + j] = acc[i][j][v];
        __syncthreads();
        for (int k = threadIdx.x; k < min(16, rt.rows - 16 * i) * (RP / 4); k += kThreads) {
            const int r = k / (RP / 4), j = k % (RP / 4) * 4;
            f32x4 s = *reinterpret_cast<const f32x4 *>(&red[0][r][j]);
#pragma unroll
            for (int v = 1; v < kWaves; ++v) s += *reinterpret_cast<const f32x4 *>(&red[v][r][j]);
            *reinterpret_cast<f32x4 *>(out + static_cast<size_t>(16 * i + r) * RP + j) = s;
        }
    }
}

// ---------------------------------------------------------------------------

struct ExpandArgs {
    const float *in;            // [parts][rows][16 RT], by place
    const uint16_t *w;          // count x cols x rank, or (LEAD) count x rank x cols
    const float *scale;
    const int32_t *order, *offsets;
    int rows, cols, rank, count, parts;
    const uint16_t *base;       // rows x cols, or null
    uint16_t *out;              // rows x cols, or null: low alone
    float *low;                 // out, rows x rank, or null
    int low_scaled;             // low with the group's scale
    int per;                    // 64-column chunks of a wave
};

// Waves of a workgroup: more share a large tile's t (2048 rows, rank 64, n 14336:
// 59 us with four in both products, 56 with eight).
constexpr int expand_waves(int mt) { return mt == 1 ? 4 : 8; }

// (Up to 32 ranks registers for four waves per SIMD, which the rare way of infinite
// sums would take: 1088 rows of 4 groups, n 2696, m 2368, rank 8, 10.7 instead of
// 12.6 us in both products.)
template <typename E, bool LEAD, int MT, int RT, bool VEC>
__global__ __launch_bounds__(64 * expand_waves(MT), RT <= 2 ? 4 : 1) void expand_kernel(const ExpandArgs a) {
    constexpr int Waves = expand_waves(MT), Threads = 64 * Waves;
    constexpr int RP = 16 * RT, Rows = 16 * MT, Units = RP / 8;
    constexpr int WF = RP < 32 ? 1 : RP / 32;  // 32-rank pieces
    constexpr int KS = RT;                     // instructions of two parts: 2 RP / 32
    constexpr int Pitch = RP + 8;
    __shared__ __attribute__((aligned(16))) uint16_t parts[2][Rows][Pitch];
    __shared__ int shifts[Rows];
    // Sums of large tiles change lanes: eight lanes take a row's 128 bytes, whole
    // lines of base and result (8192 rows, n 4096, rank 16: 59 us in both
    // products, 56 so; at 64 ranks it costs registers and with them a workgroup
    // per CU: 2048 rows, n 14336: 62 instead of 56).
    constexpr bool Turn = MT > 1 && RT != 4;
    __shared__ __attribute__((aligned(16))) float turn[Turn ? Waves : 1][Turn ? 16 : 1][Turn ? 68 : 1];
    RowTile rt;
    const int blocks = (a.cols + 64 * Waves * a.per - 1) / (64 * Waves * a.per);
    const int tile = blockIdx.x / blocks, block = blockIdx.x % blocks;
    if (!find_row_tile(a.offsets, a.count, a.rows, Rows, tile, rt)) return;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool none = rt.group >= a.count;
    const int j0 = RP < 32 ? 8 * (g & 1) : 8 * g;  // this lane's ranks of a piece

    // rows and columns of this lane's two pieces of 16 bytes of a 16 x 64 block
    int row[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!Turn && h == 1) {
                row[i][1] = row[i][0];
                continue;
            }
            const int k = 16 * i + (Turn ? 8 * h + (lane >> 3) : c), r = a.order[rt.first + min(k, rt.rows - 1)];
            row[i][h] = k < rt.rows && r >= 0 && r < a.rows ? r : -1;
        }
    auto piece = [&](int h) { return Turn ? 8 * (lane & 7) : 32 * h + 8 * g; };
    // Columns of a wave's chunk: operand 2 h + e of lane c has column 32 h + 2 c + e,
    // so that lane (c, g) gets columns 32 h + 8 g .. + 7 of row c: 16 bytes, and
    // 64 of a row in the lanes of one store.
    const uint16_t *w = a.w + static_cast<size_t>(none ? 0 : rt.group) * a.rank * a.cols;
    u32v4 wf[WF][4], base[MT][2];
    auto load = [&](int col0, auto cv, auto wv) __attribute__((always_inline)) {
        constexpr bool CV = decltype(cv)::value, WV = decltype(wv)::value;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = col0 + piece(h);
                base[m][h] = u32v4{0u, 0u, 0u, 0u};
                if (a.base && row[m][h] >= 0)
                    base[m][h] = load_row8<CV>(a.base + static_cast<size_t>(row[m][h]) * a.cols + col, a.cols - col);
            }
        if (none) return;
#pragma unroll
        for (int f = 0; f < WF; ++f) {
            if constexpr (LEAD) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t q[8][1];
                    const int col = col0 + 32 * h + 2 * c;
                    // (a rank's row from scalar registers, the lane's place in 32 bits)
                    const uint32_t at = (static_cast<uint32_t>(j0) * a.cols + col) * 2;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const char *src = reinterpret_cast<const char *>(w + static_cast<size_t>(32 * f + j) * a.cols) + at;
                        load_n<2, CV>(reinterpret_cast<const uint16_t *>(src), 32 * f + j0 + j < a.rank ? a.cols - col : 0, q[j]);
                    }
                    wf[f][2 * h] = pick_column<2>(q, 0);
                    wf[f][2 * h + 1] = pick_column<2>(q, 1);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = col0 + 32 * (i >> 1) + 2 * c + (i & 1), rk = 32 * f + j0;
                    wf[f][i] = load_row8<WV>(w + static_cast<size_t>(col) * a.rank + rk, col < a.cols ? a.rank - rk : 0);
                }
            }
        }
    };
    auto load_chunk = [&](int col0) __attribute__((always_inline)) {
        using Yes = std::true_type;
        using No = std::false_type;
        if constexpr (VEC || MT > 1) {
            using All = std::bool_constant<VEC>;
            load(col0, All{}, All{});
        } else {
            // (only the last columns of an odd width are looked at one by one; with
            // several tiles both forms cost registers: 6272 rows, n 1137, 33
            // instead of 28 us in both products)
            const bool full = col0 + 64 <= a.cols, ranks = LEAD || a.rank % 8 == 0;
            if (full && ranks) load(col0, Yes{}, Yes{});
            else if (full) load(col0, Yes{}, No{});
            else load(col0, No{}, No{});
        }
    };
    auto column = [&](int it) { return ((block * a.per + it) * Waves + wave) * 64; };
    const bool skip = !a.out || (none && a.base == a.out);
    if (!skip && column(0) < a.cols) load_chunk(column(0));  // (on its way while t is added up)

    // The tile's rows of t, once per workgroup (by each wave for itself: 2048
    // rows, rank 64, n 14336, 179 instead of 43 us): the parts added in order,
    // and the two 16-bit parts of scale * t into LDS.
    if (!none || (a.low && block == 0)) {
        const float scale = none || !a.scale ? 1.0f : a.scale[rt.group];
        for (int i = threadIdx.x; i < rt.rows * Units; i += Threads) {
            const int r = i / Units, j = i % Units * 8, at = rt.first + r;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
            if (!none) {
                const float *src = a.in + static_cast<size_t>(at) * RP + j;
                const size_t plane = static_cast<size_t>(a.rows) * RP;
                // (few rows: a wait for every eight parts, the others have each other)
                constexpr int U = MT == 1 ? 8 : 4;
                for (int p0 = 0; p0 < a.parts; p0 += U, src += U * plane) {
                    f32x4 q[U][2];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            q[u][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                            if (p0 + u < a.parts) q[u][h] = reinterpret_cast<const f32x4 *>(src + u * plane)[h];
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] += q[u][k >> 2][k & 3];
                }
            }
            if (a.low && block == 0) {
                const int to = a.order[at];
                const float by = a.low_scaled ? scale : 1.0f;
                if (to >= 0 && to < a.rows) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (j + k < a.rank) a.low[static_cast<size_t>(to) * a.rank + j + k] = v[k] * by;
                }
            }
            // (ranks behind the last: 0 where an infinite x made them 0 * inf)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = j + k < a.rank ? v[k] * scale : 0.0f;
            if constexpr (E::code == DBF_TYPE_F16) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, finite_abs(v[k]));
#pragma unroll
                for (int o = 1; o < Units; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
                const int shift = f16_shift(top);
                if (j == 0) shifts[r] = shift;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = ldexpf(v[k], shift);
            }
            u32v4 pack[2] = {pack_part<E, false>(v, 0), pack_part<E, false>(v, 1)};
            if constexpr (E::code == DBF_TYPE_BF16) {
                uint32_t odd = 0;  // (an exponent of ones: infinity, NaN, or a value above the largest)
#pragma unroll
                for (int k = 0; k < 4; ++k) odd |= ((pack[0][k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                if (__builtin_expect(odd != 0, 0)) {
                    pack[0] = pack_part<E, true>(v, 0);
                    pack[1] = pack_part<E, true>(v, 1);
                }
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) *reinterpret_cast<u32v4 *>(&parts[p][r][j]) = pack[p];
        }
    }
    __syncthreads();
    if (skip) return;
    for (int it = 0; it < a.per; ++it) {
        const int col0 = column(it);
        if (col0 >= a.cols) break;
        if (it > 0) load_chunk(col0);
        // (the weight's operands are the last of the loads; said here, or the compiler
        // waits before each store of a row's end: 256 rows of 38 groups, n 1206, m 192,
        // rank 16, 8.5 instead of 7.8 us in both products)
        wait_vm<0>();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (16 * m >= rt.rows) break;
            if (!none) {
                u32v4 tf[KS];
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    tf[s] = RP < 32 ? *reinterpret_cast<const u32v4 *>(&parts[g >> 1][16 * m + c][j0])
                                    : *reinterpret_cast<const u32v4 *>(&parts[s / WF][16 * m + c][32 * (s % WF) + j0]);
                const int shift = E::code == DBF_TYPE_F16 ? -shifts[16 * m + c] : 0;
                f32x4 acc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < KS; ++s) acc[i] = mma<E>(wf[s % WF][i], tf[s], acc[i]);
                }
                float look = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) look += (acc[i][0] + acc[i][1]) + (acc[i][2] + acc[i][3]);
                if (__builtin_expect(__ballot(16 * m + c < rt.rows && !finite(look)) != 0, 0)) {
                    // (one by one: together they cost registers, and with them a workgroup per CU)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int f = 0; f < WF; ++f) {
                            keep_order();
                            const u32v4 t = *reinterpret_cast<const u32v4 *>(&parts[0][16 * m + c][32 * f + j0]);
                            sum = mma<E>(signs<E>(wf[f][i]), signs<E>(t), sum);
                        }
                        keep_order();
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (!finite(sum[v])) acc[i][v] = sum[v];
                    }
                    keep_order();
                }
                // columns 32 h + 8 g + 2 v + e of row c, in order
                float d[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        d[h][k] = acc[2 * h + (k & 1)][k >> 1];
                        if constexpr (E::code == DBF_TYPE_F16) d[h][k] = ldexpf(d[h][k], shift);
                    }
                if constexpr (Turn) {
                    float(&own)[16][68] = turn[wave];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<f32x4 *>(&own[c][32 * h + 8 * g + 4 * q]) =
                                f32x4{d[h][4 * q], d[h][4 * q + 1], d[h][4 * q + 2], d[h][4 * q + 3]};
                    wave_fence();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const f32x4 v = *reinterpret_cast<const f32x4 *>(&own[8 * h + (lane >> 3)][8 * (lane & 7) + 4 * q]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) d[h][4 * q + k] = v[k];
                        }
                    wave_fence();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t old = base[m][h][k];
                        uint32_t o = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            o |= static_cast<uint32_t>(E::put(E::get(static_cast<uint16_t>(old >> (16 * e))) + d[h][2 * k + e])) << (16 * e);
                        base[m][h][k] = o;
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[m][h] < 0) continue;
                const int col = col0 + piece(h), valid = a.cols - col;
                uint16_t *dst = a.out + static_cast<size_t>(row[m][h]) * a.cols + col;
                if (VEC ? valid > 0 : valid >= 8) {
                    *reinterpret_cast<u32v4_any *>(dst) = base[m][h];
                } else if (!VEC) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < valid) dst[i] = static_cast<uint16_t>(base[m][h][i >> 1] >> (16 * (i & 1)));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------

// One of the two gradients: Σ over a group's rows of p (rows x rank, fp32)
// times q (rows x cols); out: count x rank x cols, or (along) count x cols x rank.
struct OuterSide {
    const float *p = nullptr;
    const uint16_t *q = nullptr;
    int cols = 0, along = 0, strips = 0;  // strips of 128 columns (0: not computed)
    const float *scale = nullptr;
    float *out = nullptr, *part = nullptr;  // part: [places of chunks][rank][cols] or [cols][rank]
};
struct OuterArgs {
    OuterSide side[2];
    const int32_t *order, *offsets;
    int rows, rank, count, chunk;  // rows of a chunk
    int most;                      // chunks in the partial sums
};

// Chunk `index` of the groups' chunks; slot: its place among the chunks of
// groups that have several, -1 for the only one of a group.  Behind the last
// chunk the groups without rows, in order (rows = 0).
__device__ __forceinline__ bool find_chunk(const OuterArgs &a, int index, RowTile &out, int &slot) {
    const int lane = threadIdx.x & 63;
    int before = 0, several = 0;
    slot = -1;
    for (int e0 = 0; e0 < a.count; e0 += 64) {
        int lo = 0, hi = 0;
        if (e0 + lane < a.count) group_places(a.offsets, a.count, a.rows, e0 + lane, lo, hi);
        const int n = (hi - lo + a.chunk - 1) / a.chunk, many = n > 1 ? n : 0;
        const int upto = before + wave_scan(n), sev = several + wave_scan(many);
        const uint64_t past = __ballot(upto > index);
        if (past) {
            const int at = __builtin_ctzll(past), i = index - __builtin_amdgcn_readlane(upto - n, at);
            out.group = e0 + at;
            out.first = __builtin_amdgcn_readlane(lo, at) + i * a.chunk;
            out.rows = min(a.chunk, __builtin_amdgcn_readlane(hi, at) - out.first);
            slot = __builtin_amdgcn_readlane(many, at) ? __builtin_amdgcn_readlane(sev - many, at) + i : -1;
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
        several = __builtin_amdgcn_readlane(sev, 63);
    }
    for (int e0 = 0; e0 < a.count; e0 += 64) {
        int lo = 0, hi = 1;
        if (e0 + lane < a.count) group_places(a.offsets, a.count, a.rows, e0 + lane, lo, hi);
        const int upto = before + wave_scan(lo == hi);
        const uint64_t past = __ballot(upto > index);
        if (past) {
            out.group = e0 + __builtin_ctzll(past);
            out.first = out.rows = 0;
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

constexpr int kMaxChunk = 2048;
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// A chunk's rows x 128 columns x 16 RT ranks per workgroup; the waves take 32
// rows in turn.
// (Registers for three workgroups per CU, which the compiler misses for f16 by
// itself: 1408 rows of 42 groups, 10688 + 768, rank 128, 169 instead of 217 us in all.)
template <typename E, int RT>
__global__ __launch_bounds__(kThreads, 3) void outer_kernel(const OuterArgs a) {
    constexpr int RP = 16 * RT, Cols = 128, Pitch = Cols + 4;
    constexpr int NP = E::code == DBF_TYPE_F16 ? 2 : 3;
    __shared__ __attribute__((aligned(16))) float sums[RP][Pitch];
    __shared__ __attribute__((aligned(16))) int rowid[kMaxChunk];
    const int strips = a.side[0].strips + a.side[1].strips;
    // (the rank blocks of a strip are neighbours on one XCD, whose L2 has its rows)
    const int rank_blocks = (a.rank + RP - 1) / RP, at = blockIdx.x % (8 * rank_blocks);
    const int work = blockIdx.x / (8 * rank_blocks) * 8 + at % 8;
    const int chunk = work / strips, st = work % strips;
    const bool second = st >= a.side[0].strips;
    const OuterSide &sd = a.side[second ? 1 : 0];
    const int strip = second ? st - a.side[0].strips : st, jb = at / 8 * RP;
    RowTile rt;
    int slot;
    if (!find_chunk(a, chunk, rt, slot)) return;
    if (slot >= a.most) return;  // (offsets that are not of an order)
    const size_t each = static_cast<size_t>(a.rank) * sd.cols;
    const int col0 = strip * Cols, nr = min(RP, a.rank - jb), nc = min(Cols, sd.cols - col0);
    float *out = slot < 0 ? sd.out + static_cast<size_t>(rt.group) * each : sd.part + static_cast<size_t>(slot) * each;
    // four neighbours of the result to memory, the first `valid` of them
    auto store4 = [](float *to, f32x4 v, int valid) {
        if (valid >= 4) {
            *reinterpret_cast<f32x4_any *>(to) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < valid) to[k] = v[k];
        }
    };
    // get(rank, column, along) of the workgroup's block, four neighbours at a time
    auto store_all = [&](auto get) {
        if (sd.along) {
            constexpr int Per = RP / 4;
            for (int i = threadIdx.x; i < Cols * Per; i += kThreads) {
                const int x = i / Per, j = i % Per * 4;
                if (x < nc) store4(out + static_cast<size_t>(col0 + x) * a.rank + jb + j, get(j, x, true), nr - j);
            }
        } else {
            constexpr int Per = Cols / 4;
            for (int i = threadIdx.x; i < RP * Per; i += kThreads) {
                const int j = i / Per, x = i % Per * 4;
                if (j < nr) store4(out + static_cast<size_t>(jb + j) * sd.cols + col0 + x, get(j, x, false), nc - x);
            }
        }
    };
    if (rt.rows == 0) {
        store_all([](int, int, bool) { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; });
        return;
    }
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = threadIdx.x; i < (rt.rows + 31) / 32 * 32; i += kThreads)
        rowid[i] = i < rt.rows ? min(max(a.order[rt.first + i], 0), a.rows - 1) : -1;
    __syncthreads();
    const int steps = (rt.rows + 31) / 32, col = col0 + 8 * c;
    const int rk = jb + c * RT;  // this lane's first rank

    // p of eight rows: ranks rk .. rk + RT - 1
    auto load_p = [&](int s, float (&p)[8][RT]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = rowid[32 * s + 8 * g + j];
            const float *src = sd.p + static_cast<size_t>(r < 0 ? 0 : r) * a.rank + rk;
#pragma unroll
            for (int i = 0; i < RT; ++i) p[j][i] = 0.0f;
            if (r < 0) continue;
            if (RT > 1 && rk + RT <= a.rank) {
                typedef float vec __attribute__((ext_vector_type(RT), aligned(4)));
                const vec v = *reinterpret_cast<const vec *>(src);
#pragma unroll
                for (int i = 0; i < RT; ++i) p[j][i] = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    if (rk + i < a.rank) p[j][i] = src[i];
            }
        }
    };
    // f16: p times 2^shift, from the largest of the wave's rows so far (sought in
    // a pass of its own: 300 rows, 1000 + 1300, rank 24, 19 instead of 22 us in all)
    int shift = E::code == DBF_TYPE_F16 ? kNoShift : 0;
    f32x4 acc[8][RT];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto turn = [&](int s, auto vec) {
        constexpr bool VEC = decltype(vec)::value;
        uint32_t q[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = rowid[32 * s + 8 * g + j];
            load_n<8, VEC>(sd.q + static_cast<size_t>(r < 0 ? 0 : r) * sd.cols + col, r < 0 ? 0 : sd.cols - col, q[j]);
        }
        float p[8][RT];
        load_p(s, p);
        if constexpr (E::code == DBF_TYPE_F16) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < RT; ++i) top = fmaxf(top, finite_abs(p[j][i]));
            top = wave_largest(top);
            const int to = top > 0.0f ? f16_shift(top) : kNoShift;
            if (to < shift) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < RT; ++j)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] = ldexpf(acc[i][j][v], to - shift);
                shift = to;
            }
        }
        u32v4 pf[RT][NP];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = E::code == DBF_TYPE_F16 ? ldexpf(p[j][i], shift) : p[j][i];
#pragma unroll
            for (int n = 0; n < NP; ++n) pf[i][n] = pack_part<E, false>(v, n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u32v4 qf = pick_column<8>(q, i);
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int n = 0; n < NP; ++n) acc[i][j] = mma<E>(qf, pf[j][n], acc[i][j]);
        }
    };
    // (only the last strip of an odd width looks at its columns one by one: 1491
    // rows, 247 + 11288, rank 128, 47 instead of 109 us)
    if (sd.cols % 8 == 0 || col0 + Cols <= sd.cols) {
        for (int s = wave; s < steps; s += kWaves) turn(s, std::true_type{});
    } else {
        for (int s = wave; s < steps; s += kWaves) turn(s, std::false_type{});
    }
    // lane (c, g): rank c RT + j, column 8 (4 g + v) + i; the waves' sums in order
    for (int w = 0; w < min(kWaves, steps); ++w) {  // (the others have no rows)
        if (wave == w) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x4 *d = reinterpret_cast<f32x4 *>(&sums[c * RT + j][32 * g + 8 * v + 4 * h]);
                        f32x4 x;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = E::code == DBF_TYPE_F16 ? ldexpf(acc[4 * h + i][j][v], -shift) : acc[4 * h + i][j][v];
                        *d = w == 0 ? x : *d + x;
                    }
        }
        __syncthreads();
    }
    const float scale = sd.scale ? sd.scale[rt.group] : 1.0f;
    float look = 0.0f;
    store_all([&](int j, int x, bool along) {
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = along ? sums[j + k][x] : sums[j][x + k];
        look += (v[0] + v[1]) + (v[2] + v[3]);
        return v * scale;
    });
    if (!__syncthreads_or(!finite(look))) return;
    // Some sum is not finite: those are stored once more, a column of each eight
    // by a wave at a time.  (In bf16 a p above the type's largest value may have
    // made them so, whose parts are taken with care here: in the loop it costs
    // 12 us of 93, 8192 rows, 4096 + 4096, rank 128.)
    for (int i = wave; i < 8; i += kWaves) {
        f32x4 sign[RT], sum[RT];
#pragma unroll
        for (int k = 0; k < RT; ++k) sign[k] = sum[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < steps; ++s) {
            float p[8][RT];
            load_p(s, p);
            u32v4 qf = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = rowid[32 * s + 8 * g + j];
                if (r >= 0 && col + i < sd.cols)
                    qf[j >> 1] |= static_cast<uint32_t>(sd.q[static_cast<size_t>(r) * sd.cols + col + i]) << (16 * (j & 1));
            }
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                float v[8];
                u32v4 pf;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = p[j][k];
#pragma unroll
                for (int j = 0; j < 4; ++j) pf[j] = sign16<E>(v[2 * j]) | sign16<E>(v[2 * j + 1]) << 16;
                sign[k] = mma<E>(signs<E>(qf), pf, sign[k]);
                if constexpr (E::code == DBF_TYPE_BF16)
#pragma unroll
                    for (int n = 0; n < NP; ++n) sum[k] = mma<E>(qf, pack_part<E, true>(v, n), sum[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int j = c * RT + k, x = 8 * (4 * g + v) + i;
                const float had = sums[j][x], now = !finite(sign[k][v]) ? sign[k][v] : E::code == DBF_TYPE_BF16 ? sum[k][v] : had;
                if (j < nr && x < nc && !finite(had))
                    out[sd.along ? static_cast<size_t>(col0 + x) * a.rank + jb + j : static_cast<size_t>(jb + j) * sd.cols + col0 + x] =
                        now * scale;
            }
    }
}

// The chunks of each group that has several, added in order.
constexpr int kJoinThreads = 64;
__global__ __launch_bounds__(kJoinThreads) void outer_join_kernel(const OuterArgs a, int blocks0) {
    const int group = blockIdx.y;
    const bool second = static_cast<int>(blockIdx.x) >= blocks0;
    const OuterSide &sd = a.side[second ? 1 : 0];
    const int block = second ? blockIdx.x - blocks0 : blockIdx.x;
    int lo, hi;
    group_places(a.offsets, a.count, a.rows, group, lo, hi);
    const int n = (hi - lo + a.chunk - 1) / a.chunk;
    if (n < 2) return;
    int first = 0;  // chunks of the groups with several before this one
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < group; e0 += 64) {
        int l = 0, h = 0;
        if (e0 + lane < group) group_places(a.offsets, a.count, a.rows, e0 + lane, l, h);
        const int k = (h - l + a.chunk - 1) / a.chunk;
        first += __builtin_amdgcn_readlane(wave_scan(k > 1 ? k : 0), 63);
    }
    const size_t each = static_cast<size_t>(a.rank) * sd.cols;
    const size_t at = (static_cast<size_t>(block) * kJoinThreads + threadIdx.x) * 4;
    if (at >= each) return;
    float *out = sd.out + static_cast<size_t>(group) * each + at;
    const float *src = sd.part + static_cast<size_t>(first) * each + at;
    const int most = min(n, a.most - first);
    if (at + 4 <= each) {
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int k = 0; k < most; ++k, src += each) v += *reinterpret_cast<const f32x4_any *>(src);
        *reinterpret_cast<f32x4_any *>(out) = v;
    } else {
        for (int i = 0; at + i < each; ++i) {
            float v = 0.0f;
            for (int k = 0; k < most; ++k) v += src[k * each + i];
            out[i] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.

int rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// 16-row tiles of a row tile: several where the groups fill them (their rows
// share the weight's operands), as many as registers and LDS allow (5400 rows, K
// 3200, rank 128: a shrink with one tile 42 us, with two 25).
constexpr int shrink_most(int rt) { return rt == 1 ? 4 : 2; }
constexpr int expand_most(int rt) { return rt == 8 ? 2 : 4; }
// (and there is enough of them for every CU: rows times the width)
bool full_groups(int rows, int count, int width) {
    return rows / (rows < count ? rows : count) >= 32 && static_cast<int64_t>(rows) * width >= 1 << 22;
}

// K parts of a shrink: about two workgroups per CU, two steps of 32 for a wave at least.
int shrink_parts(int rows, int count, int K, int rank) {
    const int64_t tiles = grouped_row_tiles(rows, count, full_groups(rows, count, K) ? 16 * shrink_most(rank_tiles(rank)) : 16);
    const int64_t steps = (K + 31) / 32, want = (512 + tiles - 1) / tiles, most = std::max<int64_t>(1, steps / (2 * kWaves));
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, kMaxParts})));
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

size_t part_bytes(int rows, int count, int K, int rank) {
    return align16(sizeof(float) * static_cast<size_t>(shrink_parts(rows, count, K, rank)) * rows * 16 * rank_tiles(rank));
}

// Rows of a chunk: enough chunks to fill the GPU, beside the half of the groups
// that may be short (1549 rows of 5 groups, 8128 + 12499, rank 32: by rows and
// columns alone 113 us in all, by ranks and groups too 89); up to 512 rows no group has several (a join's launch costs
// more than the waves' longer way).
int outer_chunk(int rows, int n, int m, int rank, int count) {
    if (rows <= 512) return 512;
    const int64_t blocks = ((n + 127) / 128 + (m + 127) / 128) * static_cast<int64_t>((rank + 31) / 32);
    int chunk = kMaxChunk;
    while (chunk > 128 && (rows / chunk + std::min(rows, count) / 2) * blocks < 1024) chunk /= 2;
    return chunk;
}
// Chunks of groups that have several: ceil(c / chunk) of more than chunk rows
// each are less than twice rows / chunk.
int64_t outer_slots(int rows, int chunk) { return rows > chunk ? 2 * static_cast<int64_t>(rows) / chunk : 0; }

template <int V>
using Tag = std::integral_constant<int, V>;
template <typename F>
void by_rank(int rank, F f) {
    switch (rank_tiles(rank)) {
        case 1: f(Tag<1>{}); break;
        case 2: f(Tag<2>{}); break;
        case 4: f(Tag<4>{}); break;
        default: f(Tag<8>{}); break;
    }
}

template <typename E, bool LEAD>
void launch_shrink(const ShrinkArgs &a, hipStream_t s) {
    by_rank(a.rank, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, Big = shrink_most(RT);
        const bool vec = a.K % 8 == 0 && (!LEAD || a.rank % RT == 0);
        auto go = [&](auto mt) {
            constexpr int MT = decltype(mt)::value;
            const dim3 grid(static_cast<uint32_t>(row_tiles_bound(a.rows, a.count, 16 * MT) * a.parts));
            if (vec) launch_kernel(shrink_kernel<E, LEAD, MT, RT, true>, grid, dim3(kThreads), 0, s, a);
            else launch_kernel(shrink_kernel<E, LEAD, MT, RT, false>, grid, dim3(kThreads), 0, s, a);
        };
        if (!full_groups(a.rows, a.count, a.K)) go(Tag<1>{});
        else go(Tag<Big>{});
    });
}

template <typename E, bool LEAD>
void launch_expand(ExpandArgs &a, hipStream_t s) {
    by_rank(a.rank, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, Big = expand_most(RT);
        const bool vec = a.cols % 8 == 0 && (LEAD || a.rank % 8 == 0);
        auto go = [&](auto mt) {
            constexpr int MT = decltype(mt)::value, Waves = expand_waves(MT), Threads = 64 * Waves;
            const int64_t tiles = row_tiles_bound(a.rows, a.count, 16 * MT);
            const int64_t chunks = (static_cast<int64_t>(a.cols) + 64 * Waves - 1) / (64 * Waves);
            // (results of t alone: one workgroup per row tile)
            a.per = static_cast<int>(a.out ? std::min<int64_t>(chunks, std::max<int64_t>(1, tiles * chunks / 512)) : chunks);
            const dim3 grid(static_cast<uint32_t>(tiles * ((chunks + a.per - 1) / a.per)));
            if (vec) launch_kernel(expand_kernel<E, LEAD, MT, RT, true>, grid, dim3(Threads), 0, s, a);
            else launch_kernel(expand_kernel<E, LEAD, MT, RT, false>, grid, dim3(Threads), 0, s, a);
        };
        if (!full_groups(a.rows, a.count, a.cols)) go(Tag<1>{});
        else go(Tag<Big>{});
    });
}

template <typename E>
void launch_outer(const OuterArgs &a, hipStream_t s) {
    // (two tiles of 16 ranks at most: four leave registers for one workgroup
    // per CU; 8192 rows, 4096 + 4096, rank 64: 163 us instead of 128 in all)
    const int rt = std::min(rank_tiles(a.rank), 2);
    const int strips = a.side[0].strips + a.side[1].strips;
    // (chunks, and groups without rows)
    const int64_t work = (static_cast<int64_t>(a.rows) / a.chunk + a.count) * strips;
    const dim3 grid(static_cast<uint32_t>((work + 7) / 8 * 8 * ((a.rank + 16 * rt - 1) / (16 * rt))));
    auto go = [&](auto r) {
        launch_kernel(outer_kernel<E, decltype(r)::value>, grid, dim3(kThreads), 0, s, a);
    };
    if (rt == 1) go(Tag<1>{});
    else go(Tag<2>{});
}

void launch_outer_join(const OuterArgs &a, hipStream_t s) {
    auto blocks = [&](const OuterSide &sd) {
        return sd.strips > 0 ? static_cast<int>((static_cast<int64_t>(a.rank) * sd.cols + 4 * kJoinThreads - 1) / (4 * kJoinThreads)) : 0;
    };
    const int b0 = blocks(a.side[0]), b1 = blocks(a.side[1]);
    launch_kernel(outer_join_kernel, dim3(b0 + b1, a.count), dim3(kJoinThreads), 0, s, a, b0);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

dbf_status_t check_sizes(int32_t type, int32_t rows, int32_t n, int32_t m, int32_t rank, int32_t count) {
    if (rows < 0 || n < 1 || m < 1 || rank < 1 || count < 1) return DBF_ERR_INVALID_ARG;
    if (type != DBF_TYPE_F16 && type != DBF_TYPE_BF16) return DBF_ERR_INVALID_ARG;
    // (a launch holds less than 2^32 threads)
    const int64_t wide = std::max(n, m);
    if (rank > kMaxRank || count > kMaxGroups || wide > (1 << 18) || rows > (1 << 24) || rows * wide > int64_t(1) << 36 ||
        int64_t(count) * rank * wide > int64_t(1) << 32)
        return DBF_ERR_SHAPE;
    return DBF_OK;
}
bool sizes_ok(int32_t rows, int32_t n, int32_t m, int32_t rank, int32_t count) {
    return check_sizes(DBF_TYPE_F16, rows, n, m, rank, count) == DBF_OK && rows > 0;
}

}  // namespace
}  // namespace dbf

extern "C" size_t dbf_adapter_workspace(int32_t rows, int32_t n, int32_t m, int32_t rank, int32_t count) {
    using namespace dbf;
    return sizes_ok(rows, n, m, rank, count) ? part_bytes(rows, count, m, rank) : 0;
}

extern "C" dbf_status_t dbf_adapter_forward(const void *x, const void *base, const void *A, const void *B,
                                            const float *scale, int32_t type, const int32_t *order,
                                            const int32_t *offsets, int32_t rows, int32_t n, int32_t m, int32_t rank,
                                            int32_t count, void *y, float *t, void *workspace, size_t workspace_bytes,
                                            hipStream_t stream) {
    using namespace dbf;
    const dbf_status_t st = check_sizes(type, rows, n, m, rank, count);
    if (st != DBF_OK || rows == 0) return st;
    for (const void *p : {x, base, A, B, static_cast<const void *>(y), static_cast<const void *>(workspace)})
        if (!p || !aligned(p, 16)) return DBF_ERR_INVALID_ARG;
    if (!order || !offsets || !aligned(order, 4) || !aligned(offsets, 4) || !aligned(scale, 4) || !aligned(t, 16) ||
        workspace_bytes < part_bytes(rows, count, m, rank))
        return DBF_ERR_INVALID_ARG;
    const size_t y_bytes = static_cast<size_t>(rows) * n * sizeof(uint16_t);
    if (y != base && share_bytes(y, y_bytes, base, y_bytes)) return DBF_ERR_INVALID_ARG;  // (other rows are read later)
    const ShrinkArgs s{static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(A), order, offsets, rows, m, rank,
                       count, shrink_parts(rows, count, m, rank), static_cast<float *>(workspace)};
    ExpandArgs e{s.out, static_cast<const uint16_t *>(B), scale, order, offsets, rows, n, rank, count, s.parts,
                 static_cast<const uint16_t *>(base), static_cast<uint16_t *>(y), t, 0, 1};
    if (type == DBF_TYPE_F16) {
        launch_shrink<F16, false>(s, stream);
        launch_expand<F16, false>(e, stream);
    } else {
        launch_shrink<BF16, false>(s, stream);
        launch_expand<BF16, false>(e, stream);
    }
    return hipGetLastError() == hipSuccess ? DBF_OK : DBF_ERR_HIP;
}

// Workspace of the backward pass: the parts of u, u, and the chunks of both gradients.
namespace {
struct BackwardPlan {
    size_t u = 0, dA = 0, dB = 0, total = 0;
};
BackwardPlan backward_plan(int32_t rows, int32_t n, int32_t m, int32_t rank, int32_t count) {
    using namespace dbf;
    BackwardPlan p;
    p.u = part_bytes(rows, count, n, rank);
    p.dA = p.u + align16(sizeof(float) * static_cast<size_t>(rows) * rank);
    const size_t slots = static_cast<size_t>(outer_slots(rows, outer_chunk(rows, n, m, rank, count)));
    p.dB = p.dA + align16(sizeof(float) * slots * rank * m);
    p.total = p.dB + align16(sizeof(float) * slots * rank * n);
    return p;
}
}  // namespace

extern "C" size_t dbf_adapter_backward_workspace(int32_t rows, int32_t n, int32_t m, int32_t rank, int32_t count) {
    return dbf::sizes_ok(rows, n, m, rank, count) ? backward_plan(rows, n, m, rank, count).total : 0;
}

extern "C" dbf_status_t dbf_adapter_backward(const void *dy, const void *x, const float *t, const void *dx,
                                             const void *A, const void *B, const float *scale, int32_t type,
                                             const int32_t *order, const int32_t *offsets, int32_t rows, int32_t n,
                                             int32_t m, int32_t rank, int32_t count, void *dx_out, float *dA, float *dB,
                                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace dbf;
    const dbf_status_t st = check_sizes(type, rows, n, m, rank, count);
    if (st != DBF_OK) return st;
    if (!dA && !dB && (!dx_out || rows == 0)) return DBF_OK;
    if (!aligned(dA, 16) || !aligned(dB, 16) || !aligned(offsets, 4) || !offsets) return DBF_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!dy || !B || !order || !workspace || (dB && !t) || (dA && !x) || (dx_out && !A)) return DBF_ERR_INVALID_ARG;
        // (dy, x and other rows of dx are read after it is written)
        const size_t x_bytes = static_cast<size_t>(rows) * m * sizeof(uint16_t);
        if (dx_out && (share_bytes(dx_out, x_bytes, dy, static_cast<size_t>(rows) * n * sizeof(uint16_t)) ||
                       (x && share_bytes(dx_out, x_bytes, x, x_bytes)) ||
                       (dx && dx_out != dx && share_bytes(dx_out, x_bytes, dx, x_bytes))))
            return DBF_ERR_INVALID_ARG;
        for (const void *p : {dy, x, dx, A, B, static_cast<const void *>(dx_out), static_cast<const void *>(workspace)})
            if (!aligned(p, 16)) return DBF_ERR_INVALID_ARG;
        if (!aligned(order, 4) || !aligned(scale, 4) || !aligned(t, 16) ||
            workspace_bytes < backward_plan(rows, n, m, rank, count).total)
            return DBF_ERR_INVALID_ARG;
    }
    const BackwardPlan plan = rows > 0 ? backward_plan(rows, n, m, rank, count) : BackwardPlan{};
    char *ws = static_cast<char *>(workspace);
    float *u = reinterpret_cast<float *>(ws + plan.u);
    if (rows > 0 && (dx_out || dA)) {
        const ShrinkArgs s{static_cast<const uint16_t *>(dy), static_cast<const uint16_t *>(B), order, offsets, rows, n,
                           rank, count, shrink_parts(rows, count, n, rank), static_cast<float *>(workspace)};
        ExpandArgs e{s.out, static_cast<const uint16_t *>(A), scale, order, offsets, rows, m, rank, count, s.parts,
                     static_cast<const uint16_t *>(dx), static_cast<uint16_t *>(dx_out), dA ? u : nullptr, 1, 1};
        if (type == DBF_TYPE_F16) {
            launch_shrink<F16, true>(s, stream);
            launch_expand<F16, true>(e, stream);
        } else {
            launch_shrink<BF16, true>(s, stream);
            launch_expand<BF16, true>(e, stream);
        }
    }
    if (dA || dB) {
        OuterArgs o{};
        o.order = order;
        o.offsets = offsets;
        o.rows = rows;
        o.rank = rank;
        o.count = count;
        o.chunk = rows > 0 ? outer_chunk(rows, n, m, rank, count) : 128;
        o.most = rows > 0 ? static_cast<int>(outer_slots(rows, o.chunk)) : 0;
        if (dA) o.side[0] = {u, static_cast<const uint16_t *>(x), m, 0, (m + 127) / 128, nullptr, dA,
                             reinterpret_cast<float *>(ws + plan.dA)};
        if (dB) o.side[1] = {t, static_cast<const uint16_t *>(dy), n, 1, (n + 127) / 128, scale, dB,
                             reinterpret_cast<float *>(ws + plan.dB)};
        if (type == DBF_TYPE_F16) launch_outer<F16>(o, stream);
        else launch_outer<BF16>(o, stream);
        if (rows > o.chunk) launch_outer_join(o, stream);
    }
    return hipGetLastError() == hipSuccess ? DBF_OK : DBF_ERR_HIP;
}
