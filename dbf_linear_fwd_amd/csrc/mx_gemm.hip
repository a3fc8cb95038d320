// Product with a 4-bit weight in blocks of 32 with power-of-two scales
// (include/dbf.h, "Block formats") on the scaled matrix-core instructions:
//   Y[b][o]  = Σ_l xq[b][l] wq[o][l]      x in e4m3 or e2m1 blocks
//
// The 32x32x64 instruction multiplies 64 columns of K per step and applies
// both operands' block scales itself.  A lane (r = lane % 32, g = lane / 32)
// supplies row r: of an e2m1 operand the 16 bytes of block g, of an e4m3
// operand bytes 16g..16g+15 of block 0 and of block 1; its scale byte is
// always that of block g.
//
// Sums are fp32, with one loss inside the instruction: e4m3 products of eight
// consecutive columns are cut off at 2^-13 of the largest of the eight.  That
// is below 2 % of what rounding that value of x into e4m3 may cost (2^-4 of
// it); 5e-6 to 6e-5 of the result where it was measured, columns up to 200
// times the others.  Exact products (x widened for the 16-bit instructions)
// run at half the rate.

#include "mx_tile.h"

namespace dbf {
namespace {

// ---------------------------------------------------------------------------
// Tiled product: a BM x BN output tile per workgroup; K goes through a ring of
// LDS stages that global_load_lds fills several stages ahead.
//
// A stage holds 64 bytes of each of the tile's rows of x (64 columns of e4m3,
// 128 of e2m1) and the weight's blocks of the same columns; scale words (four
// bytes: 128 columns) sit in stages of their own kind, one per 128 columns.
// The 16-byte chunks of a row of x are permuted so that the 16 rows which an
// operand read touches in a cycle lie on all 64 banks (as if there were 32: a
// third of the LDS cycles were conflicts, 6 % now, though the time is the
// same); the weight's and the scales' device order is the order in which the
// lanes read them.
//
// The unit of work is a half: 64 columns, MI x NI matrix-core instructions
// per wave.  While a half is multiplied, the operands of the next one are
// read from LDS and loads of a later stage are started, one or two between
// each two products: bunched in front of them they leave the matrix cores
// idle (2048 x 4096, K 14336, e4m3, 128 x 256 tiles: 104 instead of 95 us).

// A product tile: waves WM x WN, each MI x NI fragments of 32 x 32.
template <int FMT_, int MI_, int NI_, int WM_, int WN_, int S_>
struct MxTile {
    static constexpr int FMT = FMT_, MI = MI_, NI = NI_, WM = WM_, WN = WN_, S = S_;
    static constexpr bool X8 = FMT == DBF_TYPE_E4M3;
    static constexpr int Waves = WM * WN, Threads = 64 * Waves;
    static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN;
    static constexpr int Parts = X8 ? 2 : 1;               // stages per 128 columns
    static constexpr int WTile = 2048 / Parts;             // bytes of 32 weight rows in a stage
    static constexpr int XBytes = BM * 64, WBytes = BN / 32 * WTile;
    static constexpr int StageBytes = XBytes + WBytes;
    static constexpr int SBytes = (BM + BN + 63) / 64 * 256;  // scale words of x, then of w
    static constexpr int ScaleAt = S * StageBytes;            // S / Parts scale stages
    static constexpr size_t Lds = static_cast<size_t>(S) * StageBytes + static_cast<size_t>(S / Parts) * SBytes;
    static constexpr int Units16 = StageBytes / 1024;         // 1 KiB loads
    static constexpr int Units4 = SBytes / 256;               // 256-byte loads
    static constexpr int D16 = (Units16 + Waves - 1) / Waves, D4 = (Units4 + Waves - 1) / Waves;
    // loads per wave of the stage at part p of its 128 columns
    static constexpr int loads(int p) { return p == 0 ? D16 + D4 : D16; }
    // loads of the y stages after one at part p
    static constexpr int younger(int p, int y) {
        int n = 0;
        for (int i = 1; i <= y; ++i) n += loads((p + i) % Parts);
        return n;
    }
    static constexpr int XR = X8 ? 2 : 1;                     // 16-byte reads of an x fragment
    static constexpr int Reads = MI * XR + NI;
    static_assert(S % Parts == 0 && S >= 3, "whole 128 columns; a stage lands while one is read");
    static_assert(StageBytes % 1024 == 0, "whole loads");
    static_assert(Lds <= 160 * 1024, "LDS of a CU");
    static_assert(younger(0, S - 1) < 64, "vmcnt range");
};

// The operands of a half in registers.
template <typename C>
struct MxFrags {
    u32v4 x[C::MI][C::XR], w[C::NI];
};
// Scale words of 128 columns, one of four blocks for each row.
template <typename C>
struct MxScales {
    int x[C::MI], w[C::NI];
};

// Read `i` of the operands of half T from its stage.  xrow / wrow: this
// lane's place in the stage's rows of x and in its weight.
template <typename C, int T>
__device__ __forceinline__ void read_operand(const char *__restrict__ stage, MxFrags<C> &r, int i, int xrow, int wrow,
                                             int swz, int g) {
    if (i < C::MI * C::XR) {
        const int f = i / C::XR, h = i % C::XR;
        const int c = C::X8 ? 2 * h + g : 2 * T + g;
        r.x[f][h] = *reinterpret_cast<const u32v4 *>(stage + xrow + f * 2048 + ((c ^ swz) << 4));
    } else {
        const int f = i - C::MI * C::XR;
        r.w[f] = *reinterpret_cast<const u32v4 *>(stage + wrow + f * C::WTile + (C::X8 ? 0 : T * 1024));
    }
}

template <typename C>
__device__ __forceinline__ void read_scales(const char *__restrict__ stage, MxScales<C> &s, int wm, int wn, int l32) {
    const uint32_t *sc = reinterpret_cast<const uint32_t *>(stage) + l32;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) s.x[i] = static_cast<int>(sc[(wm * C::MI + i) * 32]);
#pragma unroll
    for (int f = 0; f < C::NI; ++f) s.w[f] = static_cast<int>(sc[C::BM + (wn * C::NI + f) * 32]);
}

// Bytes 0 and 2 become this lane's blocks (of lane group g) of the two halves.
template <typename C>
__device__ __forceinline__ void shift_scales(MxScales<C> &d, const MxScales<C> &s, int g) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) d.x[i] = s.x[i] >> (8 * g);
#pragma unroll
    for (int f = 0; f < C::NI; ++f) d.w[f] = s.w[f] >> (8 * g);
}

// The products of half T, with between(j) after each.
template <typename C, int T, typename F>
__device__ __forceinline__ void multiply(const MxFrags<C> &r, const MxScales<C> &s, f32x16 (&acc)[C::MI][C::NI],
                                         F between) {
    constexpr int FX = C::X8 ? 0 : 4;
    const u32v4 z = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int f = 0; f < C::NI; ++f) {
            acc[i][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                operand(r.w[f], z), operand(r.x[i][0], C::X8 ? r.x[i][C::XR - 1] : z), acc[i][f], 4, FX, 2 * T, s.w[f],
                2 * T, s.x[i]);
            between(i * C::NI + f);
            keep_order();
        }
}

// Scale rows of x (padded row layout) into 32-row tiles like the weight's: a
// step's scale words of 32 rows are 128 contiguous bytes.  Read as rows, the
// 256 words of a tile's 128 columns come from 256 cache lines (2048 x 14336,
// K 4096, e2m1: 88 instead of 83 us).
__global__ __launch_bounds__(256) void mx_tile_scales_kernel(const uint32_t *__restrict__ xs, int M, int steps,
                                                             uint32_t *__restrict__ out) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t q = idx >> 5;
    const int64_t t = q / steps;
    if (t * 32 >= M) return;
    const int k = static_cast<int>(q - t * steps);
    const int64_t row = t * 32 + (idx & 31);
    out[idx] = row < M ? xs[row * steps + k] : 0u;
}

// The same for rows in groups, by place.
__global__ __launch_bounds__(256) void mx_place_scales_kernel(const uint32_t *__restrict__ xs, const MxRows rows, int steps,
                                                              uint32_t *__restrict__ out) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t q = idx >> 5, t = q / steps;
    const int64_t place = t * 32 + (idx & 31);
    if (t * 32 >= rows.slots) return;
    if (place < rows.slots) out[idx] = xs[RowPlaces{}.in(rows, static_cast<int>(place)) * steps + (q - t * steps)];
}

struct MxGemmArgs {
    const uint8_t *xc, *xs;  // codes in padded rows; scales in 32-row tiles
    int M;
    MxWeight w;
    void *y;
    TileGrid grid;
    float *part;             // null: whole sums to y
    MxRows rows;             // grouped products
};

// G: rows in groups.  A tile's rows are those of one group, m0 = 0 its first
// and M their number.
// 2048 tokens with 2 of 8 experts each, 14336 x 4096, bf16 in e4m3: 229 us, 2.1
// PFLOP/s, matrix cores busy 55 % at a clock that falls to 1.96 GHz (4096 rows
// of one weight: 192 us).  One token, 2 of 8: 14 us, 62 MB of weights (4.4 TB/s);
// 16 tokens, 8 of 64 experts of 4096 x 1024: 22 us, 142 MB, in part from the
// last-level cache.
template <typename C, typename E, bool G>
__global__ __launch_bounds__(C::Threads) void mx_gemm_kernel(MxGemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int bm, bn, split, nsplit = a.grid.nsplit, T, tile;
    [[maybe_unused]] RowPlaces place;
    if constexpr (G) {
        const RowTiles tiles = scan_rows<C::BM>(a.rows);
        const GroupedWork w = grouped_work(tiles, a.grid.nbn, a.w.blocks >> 2, a.grid.group, nsplit, blockIdx.x);
        if (w.bm < 0) return;
        bm = w.bm;
        bn = w.bn;
        split = w.split;
        nsplit = w.nsplit;
        T = w.cut;
        tile = w.at;
        place = take_group<C::BM>(a.rows, tiles, bm, a.w, a.M);
    } else {
        T = a.grid.nbm * a.grid.nbn;
        const int idx = xcd_index(blockIdx.x, T * nsplit);
        split = idx / T;
        tile = idx - split * T;
        tile_at(a.grid, tile, bm, bn);
    }
    const int m0 = G ? 0 : bm * C::BM, n0 = bn * C::BN;
    const int lane = threadIdx.x & 63, l32 = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int steps = a.w.blocks >> 2;  // of 128 columns
    const int k0 = static_cast<int>(static_cast<int64_t>(split) * steps / nsplit);
    // (rows of no group: no steps, their results are zeros)
    const int nk = G && place.none ? 0 : static_cast<int>(static_cast<int64_t>(split + 1) * steps / nsplit) - k0;

    // sources of this wave's loads; a stage moves them by inc bytes
    const uint8_t *src[C::D16 + C::D4];
    int inc[C::D16], at[C::D16 + C::D4];
    int inc4[C::D4];
#pragma unroll
    for (int q = 0; q < C::D16; ++q) {
        const int u = min(wave * C::D16 + q, C::Units16 - 1);  // (a unit too many: loaded twice, the same bytes)
        at[q] = u * 1024;
        constexpr int XU = C::XBytes / 1024;
        if (u < XU) {
            const int c = u * 64 + lane, r = c >> 2, lc = (c & 3) ^ ((r >> 2) & 3);
            int64_t row = min(m0 + r, a.M - 1);  // rows past M: multiplied, not written
            if constexpr (G) row = place.in(a.rows, static_cast<int>(row));
            src[q] = a.xc + (static_cast<size_t>(row) * steps + k0) * (64 * C::Parts) + lc * 16;
            inc[q] = 64;
        } else {
            const int v = (u - XU) * 1024 + lane * 16;  // byte of the stage's weight
            const int t = min(n0 / 32 + v / C::WTile, a.w.n_pad / 32 - 1);
            src[q] = a.w.codes + (static_cast<size_t>(t) * steps + k0) * 2048 + v % C::WTile;
            inc[q] = C::WTile;
        }
    }
#pragma unroll
    for (int q = C::D16; q < C::D16 + C::D4; ++q) {
        const int u = min(wave * C::D4 + q - C::D16, C::Units4 - 1);
        at[q] = C::ScaleAt + u * 256;
        const int r = u * 64 + lane;
        const bool x = r < C::BM;
        // 32-row tiles; those past the end (and the padding of the last load): any valid one
        const int t = x ? min((m0 + r) / 32, (a.M + 31) / 32 - 1) : min((n0 + r - C::BM) / 32, a.w.n_pad / 32 - 1);
        src[q] = (x ? a.xs : a.w.scales) + (static_cast<size_t>(t) * steps + k0) * 128 + (r & 31) * 4;
        inc4[q - C::D16] = 128;
        if constexpr (G)
            if (x) {
                const int at = place.first + min(r, a.M - 1);
                if (a.rows.tiled) {
                    src[q] = a.xs + (static_cast<size_t>(at >> 5) * steps + k0) * 128 + (at & 31) * 4;
                } else {
                    src[q] = a.xs + (static_cast<size_t>(place.in(a.rows, at - place.first)) * steps + k0) * 4;
                    inc4[q - C::D16] = 4;
                }
            }
    }
    // load q of the stage in slot `slot`
    auto issue_one = [&](int slot, int q) {
        if (q < C::D16) {
            dma16(src[q], lds + slot * C::StageBytes + at[q]);
            src[q] += inc[q];
        } else {
            dma4(src[q], lds + (slot / C::Parts) * C::SBytes + at[q]);
            src[q] += G ? inc4[q - C::D16] : 128;
        }
    };

    f32x16 acc[C::MI][C::NI];
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int f = 0; f < C::NI; ++f)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][f][v] = 0.0f;

    const int xrow = (wm * C::MI * 32 + l32) * 64, swz = (l32 >> 2) & 3;
    const int wrow = C::XBytes + wn * C::NI * C::WTile + g * 512 + l32 * 16;
    MxFrags<C> f0, f1;
    MxScales<C> sc, sn;
    auto stage_at = [&](int slot) { return lds + slot * C::StageBytes; };
    auto scales_at = [&](int slot) { return lds + C::ScaleAt + (slot / C::Parts) * C::SBytes; };
    auto next = [](int slot) { return slot + 1 == C::S ? 0 : slot + 1; };

    // One half: multiply `cur` while `nxt` (half 1 - T of the stage in slot
    // nslot) is read and the loads of part P's stage into slot fslot start
    // (P < 0: none).  No branch inside: the compiler would move the products
    // behind it.
    constexpr int NM = C::MI * C::NI;
    auto half = [&](auto t, auto part, const MxFrags<C> &cur, MxFrags<C> &nxt, int nslot, int fslot) {
        constexpr int TC = decltype(t)::value, TN = 1 - TC, P = decltype(part)::value;
        constexpr int NL = P >= 0 ? C::loads(P) : 0;
        const char *st = stage_at(nslot);
        multiply<C, TC>(cur, sc, acc, [&](int j) {
#pragma unroll
            for (int i = C::Reads * j / NM; i < C::Reads * (j + 1) / NM; ++i)
                read_operand<C, TN>(st, nxt, i, xrow, wrow, swz, g);
            if constexpr (TN == 0)
                if (j == 0) read_scales<C>(scales_at(nslot), sn, wm, wn, l32);
#pragma unroll
            for (int q = NL * j / NM; q < NL * (j + 1) / NM; ++q) issue_one(fslot, q);
        });
        if constexpr (TN == 0) shift_scales<C>(sc, sn, g);
    };

    const int stages = nk * C::Parts;
    constexpr int Chunks = C::S / C::Parts;  // of 128 columns that the ring holds
#pragma unroll
    for (int st = 0; st < C::S; ++st)
        if (st < stages) {
#pragma unroll
            for (int q = 0; q < C::loads(st % C::Parts); ++q) issue_one(st, q);
        }
    if (nk >= Chunks) wait_vm<C::younger(0, C::S - 1)>();
    else wait_vm<0>();
    block_barrier();
#pragma unroll
    for (int i = 0; i < C::Reads; ++i) read_operand<C, 0>(stage_at(0), f0, i, xrow, wrow, swz, g);
    read_scales<C>(scales_at(0), sn, wm, wn, l32);
    shift_scales<C>(sc, sn, g);

    // Before a stage's first read: this wave's loads of it have landed, then
    // the barrier: every wave's have, and every wave's reads of the stage
    // before it have returned, so that one's slot is free for the next loads.
    // The last half reads past the last stage, in LDS and to no use.
    int slot = 0;
    auto chunk = [&](auto go, auto work) {
        constexpr bool GO = decltype(go)::value != 0, Work = decltype(work)::value != 0;
        constexpr int W0 = GO ? C::younger(0, C::S - 2) : 0, W1 = GO ? C::younger(1, C::S - 2) : 0;
        auto run = [&](auto t, auto part, const MxFrags<C> &cur, MxFrags<C> &nxt, int nslot, int fslot) {
            if constexpr (Work) {
                half(t, part, cur, nxt, nslot, fslot);
            } else {
                constexpr int P = decltype(part)::value, NL = P >= 0 ? C::loads(P) : 0;
#pragma unroll
                for (int q = 0; q < NL; ++q) issue_one(fslot, q);
            }
        };
        if constexpr (C::Parts == 2) {
            const int s1 = slot + 1, s2 = next(s1);
            wait_vm<W1>();
            wait_lds();
            block_barrier();
            run(Const<0>{}, Const<GO ? 0 : -1>{}, f0, f1, s1, slot);
            wait_vm<W0>();
            wait_lds();
            block_barrier();
            run(Const<1>{}, Const<GO ? 1 : -1>{}, f1, f0, s2, s1);
            slot = s2;
        } else {
            const int s1 = next(slot);
            run(Const<0>{}, Const<-1>{}, f0, f1, slot, 0);
            wait_vm<W0>();
            wait_lds();
            block_barrier();
            run(Const<1>{}, Const<GO ? 0 : -1>{}, f1, f0, s1, slot);
            slot = s1;
        }
    };
    auto chunks = [&](auto work) {
        int left = nk;
        for (; left > Chunks; --left) chunk(Const<1>{}, work);
        for (; left > 0; --left) chunk(Const<0>{}, work);
    };
    // Waves whose rows are all past the group's last only load: where two share
    // a SIMD, as in the largest tile, the other one has it to itself.
    if constexpr (G && C::Waves == 8) {
        if (wm * C::MI * 32 >= a.M) chunks(Const<0>{});
        else chunks(Const<1>{});
    } else {
        chunks(Const<1>{});
    }

    if (G ? nsplit > 1 : a.part != nullptr) {
        store_part<C>(part_at<C>(a.part, split, T, tile, wave, lane), acc);
        return;
    }
    static_assert(C::Waves * store_bytes<C>() <= C::Lds, "a result fits the ring");
    __syncthreads();  // every wave's last operands have been read
    if constexpr (G)
        store_tile<C, E>(lds + wave * store_bytes<C>(), acc, a.y, a.M, a.w.n, m0, n0, wave, lane,
                         [&](int r) { return place.out(a.rows, r); });
    else store_tile<C, E>(lds + wave * store_bytes<C>(), acc, a.y, a.M, a.w.n, m0, n0, wave, lane);
}

// The K parts of a tile, added in order and stored; a workgroup is one wave of
// the product's (a whole tile in one: 17 x 4096, K 14336: 16.7 instead of 15.2 us).
template <typename C, typename E, bool G>
__global__ __launch_bounds__(64) void mx_finish_kernel(MxGemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tile = blockIdx.x / C::Waves, wave = blockIdx.x % C::Waves, lane = threadIdx.x;
    constexpr size_t Each = static_cast<size_t>(C::Waves) * (C::MI * C::NI * 1024);
    f32x16 acc[C::MI][C::NI];
    if constexpr (G) {
        const RowTiles tiles = scan_rows<C::BM>(a.rows);
        const int all = tiles.work * a.grid.nbn;
        int head, parts;
        cut_tiles(all, a.w.blocks >> 2, a.grid.group, a.grid.nsplit, head, parts);
        if (tile >= all - head) return;
        GroupedWork w;
        place_tile(head + tile, a.grid.nbn, tiles.few, w);
        const RowPlaces place = take_group<C::BM>(a.rows, tiles, w.bm, a.w, a.M);
        add_parts<C>(part_at<C>(a.part, 0, all - head, tile, wave, lane), Each * (all - head), parts, acc);
        store_tile<C, E>(lds, acc, a.y, a.M, a.w.n, 0, w.bn * C::BN, wave, lane, [&](int r) { return place.out(a.rows, r); });
    } else {
        const int T = a.grid.nbm * a.grid.nbn;
        int bm, bn;
        tile_at(a.grid, tile, bm, bn);
        add_parts<C>(part_at<C>(a.part, 0, T, tile, wave, lane), Each * T, a.grid.nsplit, acc);
        store_tile<C, E>(lds, acc, a.y, a.M, a.w.n, bm * C::BM, bn * C::BN, wave, lane);
    }
}

}  // namespace

namespace {

// ---- choice of the tile and of the K parts

// A tile's cost: microseconds per 128 columns of K with few workgroups and the
// weight from HBM (a step is then as long as its loads take), and with one on
// every CU (the matrix cores' clock and the L2s are shared).  Against every
// tile and part count at 65 sizes (17 to 2048 rows, five layers of 1024 to
// 14336, both formats) the choice is 0.1 % from the best on average, 3.1 % at
// most.
struct TileCost {
    int bm, bn;
    float light[2], full[2];  // e4m3, e2m1
};
constexpr TileCost kTiles[] = {
    {256, 256, {1.30f, 0.95f}, {1.50f, 0.98f}},
    {128, 256, {0.81f, 0.60f}, {0.78f, 0.53f}},
    {128, 128, {0.60f, 0.43f}, {0.64f, 0.38f}},
    {64, 128, {0.36f, 0.30f}, {0.38f, 0.27f}},
    {64, 64, {0.28f, 0.19f}, {0.28f, 0.19f}},
    {32, 64, {0.16f, 0.16f}, {0.17f, 0.16f}},
};
constexpr int kTileCount = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr int kCus = 256;

// The tile and K parts of least estimated time: rounds of workgroups over the
// CUs, each a start of 3 us and its steps; K parts add a launch and the
// traffic of their fp32 sums.  (Ready e4m3 blocks, weight from HBM: 2048 x
// 14336, K 4096: 256 x 256 tiles 99 to 114 us, 128 x 256 117; 2048 x 4096,
// K 14336: 134 and 91; 64 x 4096, K 14336, 64 x 64 tiles: four parts 18.7, one
// 34.7; 17 x 4096, K 14336, four parts: 32 x 64 14.9, 64 x 64 17.1.)
MxPlan mx_plan(int M, int n, int steps, bool x8) {
    MxPlan best;
    float least = 0.0f;
    const int f = x8 ? 0 : 1;
    for (int t = 0; t < kTileCount; ++t) {
        const TileCost &c = kTiles[t];
        const int64_t tiles = static_cast<int64_t>((M + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn);
        for (int sp : {1, 2, 3, 4, 6, 8}) {
            if (sp > 1 && (steps < 4 * sp || tiles * sp > 2 * kCus)) break;
            const float wgs = static_cast<float>(tiles) * sp;
            const float load = wgs < kCus ? wgs / kCus : 1.0f;
            // small tiles share a CU, so their last round is only as long as it is full
            const float rounds = wgs <= kCus ? 1.0f : t < 2 ? static_cast<float>((tiles * sp + kCus - 1) / kCus) : wgs / kCus;
            const float step = c.light[f] + (c.full[f] - c.light[f]) * load;
            float us = rounds * (3.0f + static_cast<float>((steps + sp - 1) / sp) * step);
            if (sp > 1) us += 2.1f + wgs * c.bm * c.bn * 8.0f * 3.7e-7f;
            if (least == 0.0f || us < least) {
                least = us;
                best.tile = t;
                best.nsplit = sp;
            }
        }
    }
    return best;
}

// The same for rows in groups, e4m3 and e2m1.  Against every tile, cut and not,
// at 328 sizes (2 to 128 groups of 640 to 14336 by 512 to 14336, 1 to 16384 rows,
// unevenly spread, both formats) the choice is 3.5 % from the best on average, half
// of them within 1 %, at worst 61 % (16384 rows of 24 groups, 640 x 6000); by the
// costs of one weight it was 12 %: 4096 rows of 64 groups, 4096 x 1024, 62 instead
// of 47 us.
constexpr GroupedCost kGrouped[kTileCount][2] = {
    {{5.10f, 0.52f, 3.90f, 1.40f}, {4.79f, 0.38f, 4.82f, 1.02f}},
    {{4.75f, 0.50f, 7.12f, 0.81f}, {4.39f, 0.35f, 7.18f, 0.61f}},
    {{3.01f, 0.29f, 1.64f, 0.45f}, {2.68f, 0.23f, 1.94f, 0.32f}},
    {{2.38f, 0.21f, 1.94f, 0.28f}, {2.20f, 0.19f, 2.17f, 0.21f}},
    {{2.18f, 0.17f, 0.94f, 0.19f}, {1.80f, 0.14f, 1.05f, 0.13f}},
    {{2.18f, 0.14f, 1.61f, 0.12f}, {1.73f, 0.13f, 1.53f, 0.11f}},
};
// Workgroups of a tile that the GPU holds at a time: a round.
constexpr int grouped_room(int tile) { return tile == 0 ? kCus : 2 * kCus; }
constexpr int kMostParts = 8, kCutSteps = 8;
MxPlan mx_plan_grouped(int slots, int count, int n, int steps, bool x8) {
    MxPlan best;
    float least = 0.0f;
    for (int t = 0; t < kTileCount; ++t) {
        const TileCost &c = kTiles[t];
        const int64_t tiles = grouped_row_tiles(slots, count, c.bm) * ((n + c.bn - 1) / c.bn);
        for (bool cut : {false, true}) {
            if (cut && steps < kCutSteps) continue;
            const float us = grouped_estimate(kGrouped[t][x8 ? 0 : 1], tiles, steps, grouped_room(t), t == 0, kMostParts,
                                              c.bm, c.bn, cut);
            if (least == 0.0f || us < least) {
                least = us;
                best.tile = t;
                best.nsplit = cut ? kMostParts : 1;
            }
        }
    }
    return best;
}

template <int FMT, int T>
struct TileOf;
template <int FMT>
struct TileOf<FMT, 0> { using C = MxTile<FMT, 2, 4, 4, 2, FMT == DBF_TYPE_E4M3 ? 6 : 4>; };
template <int FMT>
struct TileOf<FMT, 1> { using C = MxTile<FMT, 2, 4, 2, 2, FMT == DBF_TYPE_E4M3 ? 4 : 3>; };
template <int FMT>
struct TileOf<FMT, 2> { using C = MxTile<FMT, 2, 2, 2, 2, FMT == DBF_TYPE_E4M3 ? 4 : 3>; };
template <int FMT>
struct TileOf<FMT, 3> { using C = MxTile<FMT, 2, 1, 1, 4, FMT == DBF_TYPE_E4M3 ? 8 : 6>; };
template <int FMT>
struct TileOf<FMT, 4> { using C = MxTile<FMT, 1, 1, 2, 2, FMT == DBF_TYPE_E4M3 ? 8 : 6>; };
template <int FMT>
struct TileOf<FMT, 5> { using C = MxTile<FMT, 1, 1, 1, 2, FMT == DBF_TYPE_E4M3 ? 16 : 12>; };

// The product's launch, or the join of its K parts.
template <typename C, typename E, bool G>
void launch_gemm(MxGemmArgs &a, bool join, hipStream_t s) {
    auto product = mx_gemm_kernel<C, E, G>;
    auto finish = mx_finish_kernel<C, E, G>;
    static std::atomic<uint64_t> lds_product{0};
    TileGrid &t = a.grid;
    t.nbn = (a.w.n + C::BN - 1) / C::BN;
    dim3 grid, joined;
    if constexpr (G) {
        // (the number of row tiles is on the device: the grids hold the most there can be)
        const int64_t rows = row_tiles_bound(a.M, a.rows.count, C::BM);
        grid = dim3(static_cast<uint32_t>(grouped_grid(rows, t.nbn, t.group)));
        joined = dim3(static_cast<uint32_t>(std::min<int64_t>(t.group / 2, rows * t.nbn) * C::Waves));
    } else {
        t.nbm = (a.M + C::BM - 1) / C::BM;
        t.group = t.nbm < 4 ? t.nbm : 4;
        grid = dim3(t.nbm * t.nbn * t.nsplit);
        joined = dim3(t.nbm * t.nbn * C::Waves);
    }
    if (join) {
        launch_kernel(finish, joined, dim3(64), store_bytes<C>(), s, a);
        return;
    }
    if constexpr (C::Lds > 65536) allow_lds(product, C::Lds, lds_product);
    launch_kernel(product, grid, dim3(C::Threads), C::Lds, s, a);
}

template <int FMT, typename E, bool G, int T = 0>
void launch_tile(int tile, MxGemmArgs &a, bool join, hipStream_t s) {
    if constexpr (T < kTileCount) {
        using C = typename TileOf<FMT, T>::C;
        static_assert(C::BM == kTiles[T].bm && C::BN == kTiles[T].bn, "the table's tile");
        if (tile == T) launch_gemm<C, E, G>(a, join, s);
        else launch_tile<FMT, E, G, T + 1>(tile, a, join, s);
    }
}

// Floats of the sums of a plan's K parts.
size_t part_floats(const MxPlan &p, int M, int n) {
    if (p.nsplit == 1) return 0;
    const TileCost &c = kTiles[p.tile];
    return static_cast<size_t>(p.nsplit) * ((M + c.bm - 1) / c.bm * c.bm) * ((n + c.bn - 1) / c.bn * c.bn);
}
// (a round of parts at most)
size_t grouped_part_floats(const MxPlan &p, int slots, int count, int n) {
    if (p.nsplit == 1) return 0;
    const TileCost &c = kTiles[p.tile];
    const int64_t tiles = row_tiles_bound(slots, count, c.bm) * ((n + c.bn - 1) / c.bn);
    return static_cast<size_t>(std::min<int64_t>(grouped_room(p.tile), tiles * p.nsplit)) * c.bm * c.bn;
}

int launch_either(const MxProduct &p, bool join, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.plan.nsplit > 1 && (!p.part || p.part_cap < (p.rows ? grouped_part_floats(p.plan, p.M, p.rows->count, p.w.n)
                                                              : part_floats(p.plan, p.M, p.w.n))))
        return static_cast<int>(hipErrorInvalidValue);
    MxGemmArgs a{};
    a.xc = static_cast<const uint8_t *>(p.xcodes);
    a.xs = p.xscales;
    a.M = p.M;
    a.w = p.w;
    a.y = p.y;
    a.grid.nsplit = p.plan.nsplit;
    a.part = p.plan.nsplit > 1 ? p.part : nullptr;
    if (p.rows) {
        a.rows = *p.rows;
        a.grid.group = grouped_room(p.plan.tile);
    }
    auto pick = [&](auto f) {
        constexpr int FMT = decltype(f)::value;
        if (p.rows) {
            if (p.y_type == DBF_TYPE_F16) launch_tile<FMT, F16, true>(p.plan.tile, a, join, s);
            else launch_tile<FMT, BF16, true>(p.plan.tile, a, join, s);
        } else {
            if (p.y_type == DBF_TYPE_F16) launch_tile<FMT, F16, false>(p.plan.tile, a, join, s);
            else launch_tile<FMT, BF16, false>(p.plan.tile, a, join, s);
        }
    };
    if (p.x_type == DBF_TYPE_E4M3) pick(Const<DBF_TYPE_E4M3>{});
    else pick(Const<DBF_TYPE_E2M1>{});
    return static_cast<int>(hipGetLastError());
}

}  // namespace

MxPlan mx_product_plan(int M, int n, int blocks, int x_type) {
    return mx_plan(M, n, blocks / 4, x_type == DBF_TYPE_E4M3);
}

MxPlan mx_grouped_plan(int slots, int count, int n, int blocks, int x_type) {
    return mx_plan_grouped(slots, count, n, blocks / 4, x_type == DBF_TYPE_E4M3);
}

int mx_grouped_round(const MxPlan &p) { return grouped_room(p.tile); }

size_t mx_grouped_parts(int slots, int count, int n, int blocks) {
    size_t most = 0;
    for (int t = 0; t < kTileCount && blocks / 4 >= kCutSteps; ++t)
        most = std::max(most, grouped_part_floats({t, kMostParts}, slots, count, n));
    return most;
}

void mx_product_tile(const MxPlan &p, int32_t *rows, int32_t *cols) {
    *rows = kTiles[p.tile].bm;
    *cols = kTiles[p.tile].bn;
}

size_t mx_product_parts(int M, int n, int blocks, int x_type) {
    return part_floats(mx_product_plan(M, n, blocks, x_type), M, n);
}

int launch_mx_tile_scales(const uint8_t *xs, int M, int blocks, uint8_t *out, void *stream) {
    const int steps = blocks / 4;
    const int64_t threads = static_cast<int64_t>((M + 31) / 32) * 32 * steps;
    launch_kernel(mx_tile_scales_kernel, dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0,
                  static_cast<hipStream_t>(stream), reinterpret_cast<const uint32_t *>(xs), M, steps,
                  reinterpret_cast<uint32_t *>(out));
    return static_cast<int>(hipGetLastError());
}

int launch_mx_place_scales(const uint8_t *xs, const MxRows &rows, int blocks, uint8_t *out, void *stream) {
    const int steps = blocks / 4;
    const int64_t threads = static_cast<int64_t>((rows.slots + 31) / 32) * 32 * steps;
    launch_kernel(mx_place_scales_kernel, dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0,
                  static_cast<hipStream_t>(stream), reinterpret_cast<const uint32_t *>(xs), rows, steps,
                  reinterpret_cast<uint32_t *>(out));
    return static_cast<int>(hipGetLastError());
}

int launch_mx_product(const MxProduct &p, void *stream) { return launch_either(p, false, stream); }

int launch_mx_product_join(const MxProduct &p, void *stream) { return launch_either(p, true, stream); }

}  // namespace dbf
