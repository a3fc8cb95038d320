// Gradient of the input through a 4-bit block weight:
//   dX[b][l] = Σ_o dy[b][o] w[o][l],   dy and dX in f16 or bf16.
//
// The sum runs over the weight's rows, across its blocks, so every term of a
// sum has another scale and the scaled matrix-core instructions do not apply:
// the weight becomes 16-bit values on the way, on the 32x32x16 instructions
// (2.5 PFLOP/s).  Per 64 rows of the weight a thread takes one block (one row,
// 32 columns) and widens its codes relative to the largest scale of their
// block column, code * 2^(s - smax + kShift), into LDS; the transposing LDS read
// hands a lane the rows of its column.  f16 holds the codes exactly down to
// scales of 2^-36 of the largest (0.5 is 2^-24 then), bf16 to 2^-125; smaller
// ones lose bits or vanish.  The sums are multiplied by 2^(smax - kShift) at
// the end.  (As bytes in LDS, e5m2 of the same values, widened again by every
// wave that reads them: 243 us where this took 237.)
//
// 2048 rows, n 14336, m 4096, bf16: 205 to 225 us as the clock goes, 1.07 to
// 1.17 PFLOP/s (a library product of 16-bit matrices of that size takes 211);
// n 14344, no whole steps, 217 to 234; n 14337, rows that are not 16-byte
// aligned and go through registers, 612.  A step of 64 rows of a 256 x 256 tile
// takes 1.25 us alone and 1.8 with all CUs at work, where the clock falls to
// 1.9 GHz; its products are 0.85 us at the highest clock.

#include "mx_tile.h"

namespace dbf {
namespace {

// Exponent that the largest scale of a block column stands at: in f16 the
// largest code, 6 * 2^13, is within the type and the small ones reach furthest
// down; bf16 has fp32's range, and a sum overflows where dy's own does.
template <typename E>
constexpr int kShift = E::code == DBF_TYPE_F16 ? 13 : 0;

// Waves WM x WN, each MI x NI fragments of 32 x 32.
template <int MI_, int NI_, int WM_, int WN_>
struct GradTile {
    static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = WN_;
    static constexpr int Waves = WM * WN, Threads = 64 * Waves;
    static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN, BK = 64;
    static constexpr int ABytes = BM * BK * 2;
    static constexpr int BPitch = BN * 2;  // bytes of a weight row
    static constexpr int BBytes = BK * BPitch;
    static constexpr int AStages = 2, BStages = 2, RStages = 2;
    static constexpr int NB = BN / 32 * BK / Threads;  // weight blocks per thread and step
    static constexpr int RBytes = NB * 1280;           // a wave's codes and scale words of a step
    static constexpr int BAt = AStages * ABytes, RAt = BAt + BStages * BBytes;
    static constexpr size_t Lds = static_cast<size_t>(RAt) + static_cast<size_t>(RStages) * Waves * RBytes;
    static constexpr int DA = ABytes / 1024 / Waves;  // 1 KiB loads per wave and step
    static_assert(NB * Threads == BN / 32 * BK, "whole blocks per thread");
    static_assert(DA * Waves * 1024 == ABytes, "whole loads");
    static_assert(Lds <= 160 * 1024, "LDS of a CU");
    static_assert(static_cast<size_t>(Waves) * 32 * (64 * NI + 16) <= Lds, "a result fits");
};

struct MxGradArgs {
    const void *dy;
    const void *zeros;  // 16 zero bytes
    int M;
    MxWeight w;
    void *dx;
    TileGrid grid;
    float *part;
};

// The factor of a block's codes: 2^(s - smax + kShift).
template <typename E>
__device__ __forceinline__ float block_scale(int s, int smax) {
    const int e = 127 + kShift<E> - smax + s;
    const uint32_t bits = s == 255 ? 0x7fc00000u : static_cast<uint32_t>(e > 0 ? e : 0) << 23;
    return __builtin_bit_cast(float, bits);
}

// Eight codes as 16-bit values times sc.
template <typename E>
__device__ __forceinline__ u32v4 widen(uint32_t w, float sc) {
    u32v4 r;
    if constexpr (E::code == DBF_TYPE_BF16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 3));
    }
    return r;
}

// Transposing read of 4 x 16 16-bit values by 16 lanes.  (The restrict-qualified
// argument keeps the compiler from waiting for every load into LDS first.)
__device__ __forceinline__ u32v2 read_columns(const char *__restrict__ p) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s4;
    return __builtin_bit_cast(u32v2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p));
}

// A lane's codes and scale word of a block.
__device__ __forceinline__ void read_raw(const char *__restrict__ p, int lane, u32v4 &codes, uint32_t &scales) {
    codes = *reinterpret_cast<const u32v4 *>(p + lane * 16);
    scales = *reinterpret_cast<const uint32_t *>(p + 1024 + lane * 4);
}

template <typename E>
__device__ __forceinline__ f32x16 product(u32v4 w, u32v4 d, f32x16 acc) {
    if constexpr (E::code == DBF_TYPE_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, d), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, d), acc, 0, 0, 0);
}

// The sums times 2^(smax - kShift) of their block column.
template <typename C, typename E>
__device__ __forceinline__ void scale_columns(f32x16 (&acc)[C::MI][C::NI], const MxWeight &w, int n0, int wn) {
#pragma unroll
    for (int f = 0; f < C::NI; ++f) {
        const int kb = min(n0 / 32 + wn * C::NI + f, w.blocks - 1);
        const int e = static_cast<int>(w.colmax[kb]) - 127 - kShift<E>;
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][f][v] = ldexpf(acc[i][f][v], e);
    }
}

// How dy and the weight are read.  Whole: n is a multiple of 64, so every step
// is whole and its addresses are a common base and a lane's constant offset
// (2048 rows, n 14336, m 4096: 209 us; with a check for the last columns and
// rows in each step, at n 14344, 217).  Rows16: dy's rows are 16-byte aligned
// (n a multiple of 8).  Elements: any n, dy through registers.
enum class GradRows { Whole, Rows16, Elements };

template <typename C, typename E, GradRows ROWS>
__global__ __launch_bounds__(C::Threads) void mx_grad_kernel(const MxGradArgs a) {
    constexpr bool Whole = ROWS == GradRows::Whole, Dma = ROWS != GradRows::Elements;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int T = a.grid.nbm * a.grid.nbn;
    const int idx = xcd_index(blockIdx.x, T * a.grid.nsplit);
    const int split = idx / T, tile = idx - split * T;
    int bm, bn;
    tile_at(a.grid, tile, bm, bn);
    const int m0 = bm * C::BM, n0 = bn * C::BN;
    const int lane = threadIdx.x & 63, l32 = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int steps = (a.w.n + C::BK - 1) / C::BK;
    const int k0 = static_cast<int>(static_cast<int64_t>(split) * steps / a.grid.nsplit);
    const int nk = static_cast<int>(static_cast<int64_t>(split + 1) * steps / a.grid.nsplit) - k0;
    const uint16_t *dy = static_cast<const uint16_t *>(a.dy);

    // dy: chunk c of eight columns of row r sits at position c ^ (r & 7)
    const uint16_t *src[C::DA];
    uint32_t off[C::DA];  // Whole: bytes from the tile's first row and the step's first column
    int col[C::DA];
#pragma unroll
    for (int q = 0; q < C::DA; ++q) {
        const int c = (wave * C::DA + q) * 64 + lane, r = c >> 3, at = ((c & 7) ^ ((r >> 1) & 7)) * 8;
        const int row = min(m0 + r, a.M - 1);  // rows past M: not written
        col[q] = k0 * C::BK + at;
        src[q] = dy + static_cast<size_t>(row) * a.w.n + col[q];
        off[q] = (static_cast<uint32_t>(row - m0) * a.w.n + at) * 2;
    }
    const char *tile_dy = reinterpret_cast<const char *>(dy + static_cast<size_t>(m0) * a.w.n);
    int dstep = k0;  // of load_dy's next call
    auto load_dy = [&](int slot) {  // the next step's, each call
        char *st = lds + slot * C::ABytes;
#pragma unroll
        for (int q = 0; q < C::DA; ++q) {
            if constexpr (Whole) {
                dma16(tile_dy + static_cast<size_t>(min(dstep, steps - 1)) * (2 * C::BK) + off[q],
                      st + (wave * C::DA + q) * 1024);
            } else if constexpr (Dma) {
                // columns past n: zeros, whatever stands in the next row
                dma16(col[q] < a.w.n ? static_cast<const void *>(src[q]) : a.zeros, st + (wave * C::DA + q) * 1024);
            } else {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = col[q] + 2 * i < a.w.n ? src[q][2 * i] : 0;
                    const uint32_t y = col[q] + 2 * i + 1 < a.w.n ? src[q][2 * i + 1] : 0;
                    v[i] = x | y << 16;
                }
                *reinterpret_cast<u32v4 *>(st + (wave * C::DA + q) * 1024 + lane * 16) = u32v4{v[0], v[1], v[2], v[3]};
            }
            if constexpr (!Whole) {
                src[q] += C::BK;
                col[q] += C::BK;
            }
        }
        ++dstep;
    };
    // weight: this thread's blocks are row `lane` of the step, block columns
    // n0 / 32 + NB wave + i
    int kb[C::NB], smax[C::NB];
#pragma unroll
    for (int i = 0; i < C::NB; ++i) {
        kb[i] = min(n0 / 32 + wave * C::NB + i, a.w.blocks - 1);  // block columns past the end: not written
        smax[i] = __builtin_amdgcn_readfirstlane(a.w.colmax[kb[i]]);
    }
    int wrow = k0 * C::BK + lane;  // of the step that take_w takes next
    int lrow = wrow;               // of the step that load_w takes next
    int lstep = k0;
    const uint32_t woff = static_cast<uint32_t>(lane >> 5) * a.w.blocks * 512 + (lane & 31) * 16;
    const uint32_t soff = static_cast<uint32_t>(lane >> 5) * (a.w.blocks >> 2) * 128 + (lane & 31) * 4;
    // Through LDS too, each wave its own (loaded into registers, they would
    // have the compiler wait for every load that is under way).
    auto load_w = [&](int slot) {
        char *p = lds + C::RAt + (slot * C::Waves + wave) * C::RBytes;
        if constexpr (Whole) {
            const size_t t = 2 * static_cast<size_t>(min(lstep, steps - 1));
#pragma unroll
            for (int i = 0; i < C::NB; ++i) {
                dma16(a.w.codes + (t * a.w.blocks + kb[i]) * 512 + woff, p + i * 1280);
                dma4(a.w.scales + (t * (a.w.blocks >> 2) + (kb[i] >> 2)) * 128 + soff, p + i * 1280 + 1024);
            }
            ++lstep;
        } else {
            const int row = min(lrow, a.w.n_pad - 1);
            const size_t t = static_cast<size_t>(row >> 5);
#pragma unroll
            for (int i = 0; i < C::NB; ++i) {
                dma16(a.w.codes + ((t * a.w.blocks + kb[i]) * 32 + (row & 31)) * 16, p + i * 1280);
                dma4(a.w.scales + ((t * (a.w.blocks >> 2) + (kb[i] >> 2)) * 32 + (row & 31)) * 4, p + i * 1280 + 1024);
            }
            lrow += C::BK;
        }
    };
    constexpr int DW = 2 * C::NB;  // loads of a step's weight
    u32v4 wcodes[C::NB];
    float wscale[C::NB];
    uint32_t wsw[C::NB];
    auto read_w = [&](int slot) {
        const char *p = lds + C::RAt + (slot * C::Waves + wave) * C::RBytes;
#pragma unroll
        for (int i = 0; i < C::NB; ++i) read_raw(p + i * 1280, lane, wcodes[i], wsw[i]);
    };
    auto take_w = [&] {
        const bool past = !Whole && wrow >= a.w.n;  // rows past n are zeros
#pragma unroll
        for (int i = 0; i < C::NB; ++i) {
            const int sb = static_cast<int>(wsw[i] >> (8 * (kb[i] & 3)) & 255u);
            if (past) wcodes[i] = u32v4{0u, 0u, 0u, 0u};
            wscale[i] = block_scale<E>(past ? 0 : sb, smax[i]);
        }
        wrow += C::BK;
    };
    // The weight's values: 16-byte chunk c (of 16) of each 256 bytes of row r
    // sits at c ^ (4 (r % 4) + r / 4 % 4): what 16 lanes write, and the four
    // rows that 32 lanes of a transposing read touch, lie on all 64 banks.
    const int bswz = ((lane & 3) << 2) | ((lane >> 2) & 3);
    auto put_w = [&](int bslot, int j) {  // eight columns of each block
#pragma unroll
        for (int i = 0; i < C::NB; ++i) {
            const int blk = wave * C::NB + i;
            *reinterpret_cast<u32v4 *>(lds + C::BAt + bslot * C::BBytes + lane * C::BPitch + (blk >> 2) * 256 +
                                       ((((blk & 3) * 4 + j) ^ bswz) << 4)) = widen<E>(wcodes[i][j], wscale[i]);
        }
    };

    f32x16 acc[C::MI][C::NI];
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int f = 0; f < C::NI; ++f)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][f][v] = 0.0f;

    // operands of 16 rows of the weight
    struct Frags {
        u32v4 d[C::MI], w[C::NI];
    };
    const int arow = (wm * C::MI * 32 + l32) * 128;
    // transposing read h of an operand: lane i of 16 gives row 8 g + 4 h + i / 4,
    // four columns; gets column i, four rows
    int bat[C::NI][2];
#pragma unroll
    for (int j = 0; j < C::NI; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane & 15, blk = wn * C::NI + j, c = (blk & 3) * 4 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
            bat[j][h] = C::BAt + (8 * g + 4 * h + (i >> 2)) * C::BPitch + (blk >> 2) * 256 +
                        ((c ^ (((i >> 2) << 2) | ((2 * g + h) & 3))) << 4) + (i & 1) * 8;
        }
    auto load_frags = [&](int ks, int aslot, int bslot, Frags &f) {
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const u32v2 lo = read_columns(lds + bat[j][0] + bslot * C::BBytes + ks * 16 * C::BPitch);
            const u32v2 hi = read_columns(lds + bat[j][1] + bslot * C::BBytes + ks * 16 * C::BPitch);
            f.w[j] = u32v4{lo[0], lo[1], hi[0], hi[1]};
            if (j == 0) {
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
                    f.d[i] = *reinterpret_cast<const u32v4 *>(lds + aslot * C::ABytes + arow + i * 4096 +
                                                              (((2 * ks + g) ^ ((l32 >> 1) & 7)) << 4));
            }
        }
    };
    auto multiply = [&](const Frags &f) {
#pragma unroll
        for (int j = 0; j < C::NI; ++j)
#pragma unroll
            for (int i = 0; i < C::MI; ++i) acc[i][j] = product<E>(f.w[j], f.d[i], acc[i][j]);
    };
    // Order of a region: its LDS reads behind the first products, two vector
    // instructions after each.
    auto interleave = [&] {
#pragma unroll
        for (int i = 0; i < C::MI * C::NI; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
        keep_order();
    };

    // Step kt: dy and the weight's values in slots kt % 2.  Under way: dy of step
    // kt + 1, the weight's codes of steps kt + 1 and kt + 2 (slots kt % 2
    // again).  The operands of each of its four times 16 rows are read beside the
    // products before; the next step's weight is converted beside the first
    // three, its codes read before them.  The loads run on past the last step, to
    // no use: a branch around them would have the compiler move the products
    // behind it.
    Frags f0, f1;
    load_w(0);
    load_w(1);
    load_dy(0);
    wait_vm<(Dma ? C::DA : 0) + DW>();
    read_w(0);
    take_w();
#pragma unroll
    for (int j = 0; j < 4; ++j) put_w(0, j);
    keep_order();  // (step 0's codes have been read)
    load_w(0);
    load_dy(1);
    wait_vm<(Dma ? C::DA : 0) + DW>();
    wait_lds();
    block_barrier();
    load_frags(0, 0, 0, f0);
    read_w(1);
    int s = 0;
    for (int kt = 0; kt < nk; ++kt) {
        load_frags(1, s, s, f1);
        multiply(f0);
        take_w();
        put_w(s ^ 1, 0);
        interleave();
        load_w(s ^ 1);
        keep_order();
        load_frags(2, s, s, f0);
        multiply(f1);
        put_w(s ^ 1, 1);
        put_w(s ^ 1, 2);
        interleave();
        load_frags(3, s, s, f1);
        multiply(f0);
        put_w(s ^ 1, 3);
        interleave();
        // The next step's dy and the codes behind it have landed (younger: a
        // step's codes).  Past the barrier that holds for every wave, the next
        // step's weight is in LDS, and this step's operands have been read.
        wait_vm<DW>();
        wait_lds();
        block_barrier();
        load_frags(0, s ^ 1, s ^ 1, f0);
        read_w(s);
        load_dy(s);
        multiply(f1);
        interleave();
        s ^= 1;
    }
    wait_vm<0>();  // nothing more lands in the LDS that the result goes through
    wait_lds();
    block_barrier();

    if (a.part) {
        store_part<C>(part_at<C>(a.part, split, T, tile, wave, lane), acc);
        return;
    }
    scale_columns<C, E>(acc, a.w, n0, wn);
    store_tile<C, E>(lds + wave * store_bytes<C>(), acc, a.dx, a.M, a.w.m, m0, n0, wave, lane);
}

template <typename C, typename E>
__global__ __launch_bounds__(64) void mx_grad_finish_kernel(const MxGradArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int T = a.grid.nbm * a.grid.nbn, tile = blockIdx.x / C::Waves, wave = blockIdx.x % C::Waves;
    int bm, bn;
    tile_at(a.grid, tile, bm, bn);
    const int lane = threadIdx.x;
    f32x16 acc[C::MI][C::NI];
    add_parts<C>(part_at<C>(a.part, 0, T, tile, wave, lane), static_cast<size_t>(T) * C::Waves * (C::MI * C::NI * 1024),
                 a.grid.nsplit, acc);
    scale_columns<C, E>(acc, a.w, bn * C::BN, wave % C::WN);
    store_tile<C, E>(lds, acc, a.dx, a.M, a.w.m, bm * C::BM, bn * C::BN, wave, lane);
}

// ---- choice of the tile and of the K parts

// A tile's cost in microseconds per 64 rows of the weight: with few
// workgroups (a step's latency), and per workgroup of a full CU.  Measured at
// n 14336, m 4096 and n 4096, m 14336.
struct GradCost {
    int bm, bn;
    float light, full;
};
constexpr GradCost kGrad[] = {
    {256, 256, 1.20f, 1.85f},
    {128, 128, 0.64f, 0.66f},
    {32, 128, 0.46f, 0.29f},
};
constexpr int kGradCount = sizeof(kGrad) / sizeof(kGrad[0]);
constexpr int kCus = 256;

// The tile and K parts of least estimated time; K parts add a launch and the
// traffic of their fp32 sums.  (n 14336, m 4096, bf16, weight from HBM: 2048
// rows in 256 x 256 tiles and two parts 206 us, whole 288, 128 x 128 tiles 242;
// 1024 rows in four parts 116, 128 x 128 tiles in two 136; 16 rows in 32 x 128
// tiles and twelve parts 21.7, whole 100.  Parts are priced too high: at 35
// sizes the choice is 4.4 % from the best on average; 512 rows take 88 us in
// 128 x 128 tiles and two parts, 77.5 in 256 x 256 and eight; at worst 45.5
// where 35 is the best, 128 rows of n 4096, m 14336.)
MxPlan grad_plan(int M, int n, int m) {
    MxPlan best;
    float least = 0.0f;
    const int steps = (n + 63) / 64;
    for (int t = 0; t < kGradCount; ++t) {
        const GradCost &c = kGrad[t];
        const int64_t tiles = static_cast<int64_t>((M + c.bm - 1) / c.bm) * ((m + c.bn - 1) / c.bn);
        for (int sp : {1, 2, 3, 4, 6, 8, 12}) {
            if (sp > 1 && (steps < 4 * sp || tiles * sp > 2 * kCus)) break;
            const float wgs = static_cast<float>(tiles) * sp;
            // the largest tile has a CU to itself; smaller ones share
            const float per_cu = t == 0 ? static_cast<float>((tiles * sp + kCus - 1) / kCus) : wgs / kCus;
            const float step = c.full * per_cu > c.light ? c.full * per_cu : c.light;
            float us = 3.0f + static_cast<float>((steps + sp - 1) / sp) * step;
            if (sp > 1) us += 3.5f + wgs * c.bm * c.bn * 8.0f * 3e-7f;
            if (least == 0.0f || us < least) {
                least = us;
                best.tile = t;
                best.nsplit = sp;
            }
        }
    }
    return best;
}

// The product's launch, or the join of its K parts.
template <typename C, typename E>
void launch_grad(MxGradArgs &a, bool join, hipStream_t s) {
    static std::atomic<uint64_t> lds0{0}, lds1{0}, lds2{0};
    TileGrid &t = a.grid;
    t.nbm = (a.M + C::BM - 1) / C::BM;
    t.nbn = (a.w.m + C::BN - 1) / C::BN;
    t.group = t.nbm < 4 ? t.nbm : 4;
    if (join) {
        auto k = mx_grad_finish_kernel<C, E>;
        launch_kernel(k, dim3(t.nbm * t.nbn * C::Waves), dim3(64), store_bytes<C>(), s, a);
        return;
    }
    const dim3 grid(t.nbm * t.nbn * t.nsplit);
    auto go = [&](auto rows, std::atomic<uint64_t> &asked) {
        auto k = mx_grad_kernel<C, E, decltype(rows)::value>;
        if constexpr (C::Lds > 65536) allow_lds(k, C::Lds, asked);
        launch_kernel(k, grid, dim3(C::Threads), C::Lds, s, a);
    };
    // (offsets inside a tile are 32 bits)
    if (a.w.n % C::BK == 0 && a.w.n <= 1 << 22 && a.w.blocks <= 1 << 22)
        go(std::integral_constant<GradRows, GradRows::Whole>{}, lds0);
    else if (a.w.n % 8 == 0) go(std::integral_constant<GradRows, GradRows::Rows16>{}, lds1);
    else go(std::integral_constant<GradRows, GradRows::Elements>{}, lds2);
}

// Floats of the sums of a plan's K parts.
size_t part_floats(const MxPlan &p, int M, int m) {
    if (p.nsplit == 1) return 0;
    const GradCost &c = kGrad[p.tile];
    return static_cast<size_t>(p.nsplit) * ((M + c.bm - 1) / c.bm * c.bm) * ((m + c.bn - 1) / c.bn * c.bn);
}

int launch_either(const MxBackward &b, bool join, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (b.plan.nsplit > 1 && (!b.part || b.part_cap < part_floats(b.plan, b.M, b.w.m)))
        return static_cast<int>(hipErrorInvalidValue);
    MxGradArgs a{};
    a.dy = b.dy;
    a.zeros = b.zeros;
    a.M = b.M;
    a.w = b.w;
    a.dx = b.dx;
    a.grid.nsplit = b.plan.nsplit;
    a.part = b.plan.nsplit > 1 ? b.part : nullptr;
    auto go = [&](auto e) {
        using E = decltype(e);
        if (b.plan.tile == 0) launch_grad<GradTile<4, 2, 2, 4>, E>(a, join, s);
        else if (b.plan.tile == 1) launch_grad<GradTile<2, 2, 2, 2>, E>(a, join, s);
        else launch_grad<GradTile<1, 1, 1, 4>, E>(a, join, s);
    };
    if (b.type == DBF_TYPE_BF16) go(BF16{});
    else go(F16{});
    return static_cast<int>(hipGetLastError());
}

}  // namespace

MxPlan mx_backward_plan(int M, int n, int m) { return grad_plan(M, n, m); }

void mx_backward_tile(const MxPlan &p, int32_t *rows, int32_t *cols) {
    *rows = kGrad[p.tile].bm;
    *cols = kGrad[p.tile].bn;
}

size_t mx_backward_parts(int M, int n, int m) { return part_floats(grad_plan(M, n, m), M, m); }

int launch_mx_backward(const MxBackward &b, void *stream) { return launch_either(b, false, stream); }

int launch_mx_backward_join(const MxBackward &b, void *stream) { return launch_either(b, true, stream); }

}  // namespace dbf
