// Products with a 4-bit block weight for few rows (batch 1..16).
//
// The weight's bytes are all there is to move, so the kernel streams them
// once: K is cut between the eight waves of a workgroup, and a workgroup goes
// through its tiles of 16 output rows, of one or several layers that share x.
// A wave multiplies 16 weight rows x 128 columns with the rows of x per
// matrix-core instruction (the weight as the first operand, the batch as the
// second one's columns; a batch of one costs the same as 16).  The waves' sums
// of a tile meet in LDS and are added in wave order, while the next tile's
// weight is on its way.
//
// Of the 16x16x128 instruction a lane (c = lane % 16, g = lane / 16) supplies
// row c: of an e2m1 operand the 16 bytes of block g; of an e4m3 operand bytes
// 16 g .. of the first 64 columns and of the second 64.  Its scale byte is
// block g's either way.
//
// x goes through LDS.  Up to 65536 values of 16 bits are quantised on the way,
// without a launch of their own, while the first weight tile is coming: all
// threads of a workgroup together, two lanes per block.  (By each wave in its
// operand registers, where the lanes of absent batch rows repeat the work:
// batch 1, 4096 x 14336: 13.1 instead of 10.3 us.)  More of them are better
// quantised once than in every workgroup, at 2.5 us for the launch: 16 x 8192
// for 8192 rows 16.1 and 16.8 us, 16 x 14336 in e2m1 for 4096 rows 14.9 and
// 21.8; 16 x 4096 for 4096 rows 8.7 and 7.8.
// Batches whose blocks do not fit LDS go to the tiled product (read from L2
// for every tile, 16 x 14336 for 4096 rows took 17 us where the tiles took 13).
//
// Graph replays with weights from HBM: 14336 x 4096 at batch 1 9.3 us (3.4
// TB/s; a large copy reaches 4.6; 7.5 from the last-level cache), batch 16,
// quantising included, 12.9; 4096 x 14336 at batch 1 10.6 us (one tile per
// workgroup: nothing to overlap with x's way to LDS); 4096 x 4096 5.2 us;
// 1024 x 4096 4.5 us; three layers of 4096, 1024 and 1024 rows that share 4096
// columns 6.5 us in one launch, 14.3 in three.

#include "mx_tile.h"

namespace dbf {
namespace {

// Rows of x as the kernel's template argument: 16-bit values, or ready blocks.
constexpr int kBlocks = -1;

// Largest magnitude of 16-bit values, two per word: sign bits off, as integers.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t absmax(u32v4 a, u32v4 b) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = a[i] & 0x7fff7fffu, q = b[i] & 0x7fff7fffu;
        m = max16x2(m, max16x2(p, q));
    }
    return m;
}
// Float bits of the larger half of a word of 16-bit magnitudes.
template <int XT>
__device__ __forceinline__ uint32_t float_bits(uint32_t m) {
    const uint32_t h = m >> 16, l = m & 0xffffu, v = h > l ? h : l;
    if constexpr (XT == DBF_TYPE_BF16) return v << 16;
    else return __builtin_bit_cast(uint32_t, F16::get(static_cast<uint16_t>(v)));
}

// Codes of 16 values (two words of eight each at a and b): e4m3 in four
// words, e2m1 in two.  Under mx_saturate.
template <int XT, int ACT>
__device__ __forceinline__ u32v4 codes16(u32v4 a, u32v4 b, float sc) {
    u32v4 r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = i < 4 ? a[i & 3] : b[i & 3];
        if constexpr (ACT == DBF_TYPE_E4M3) {
            const uint32_t old = r[i >> 1];
            s16x2 o = __builtin_bit_cast(s16x2, old);
            if constexpr (XT == DBF_TYPE_BF16) {
                const bf16x2 v = __builtin_bit_cast(bf16x2, w);
                o = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, sc, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, sc, false);
            } else {
                const f16x2 v = __builtin_bit_cast(f16x2, w);
                o = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(o, v, sc, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(o, v, sc, false);
            }
            r[i >> 1] = __builtin_bit_cast(uint32_t, o);
        } else {
            uint32_t o = r[i >> 2];
            auto put = [&](auto sel) {
                constexpr int S = decltype(sel)::value;
                if constexpr (XT == DBF_TYPE_BF16) o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w), sc, S);
                else o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(o, __builtin_bit_cast(f16x2, w), sc, S);
            };
            switch (i & 3) {
                case 0: put(std::integral_constant<int, 0>{}); break;
                case 1: put(std::integral_constant<int, 1>{}); break;
                case 2: put(std::integral_constant<int, 2>{}); break;
                default: put(std::integral_constant<int, 3>{}); break;
            }
            r[i >> 2] = o;
        }
    }
    return r;
}

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// x in LDS: rows of codes and of scale bytes, their pitches off a multiple of
// the banks so that the rows of an operand read fall on different ones.
template <int ACT>
struct XLds {
    __host__ __device__ static int row_bytes(int blocks) { return blocks * (ACT == DBF_TYPE_E4M3 ? 32 : 16); }
    __host__ __device__ static int code_pitch(int blocks) { return row_bytes(blocks) + 16; }
    __host__ __device__ static int scale_pitch(int blocks) { return blocks + 4; }
    static size_t bytes(int batch, int blocks) {
        return static_cast<size_t>(batch) * (code_pitch(blocks) + scale_pitch(blocks));
    }
};
constexpr size_t kSumBytes = 2 * kWaves * 64 * 16;
constexpr size_t kMaxXBytes = 160 * 1024 - kSumBytes;

// XT: type of x's rows (f16, bf16) or kBlocks; SPW: steps of 128 columns of a
// wave at most.
template <int XT, int ACT, typename E, int SPW>
__global__ __launch_bounds__(kThreads, 4) void mx_decode_kernel(const MxDecodeArgs a) {
    // units of a thread in flight while x goes to LDS (registers for two workgroups per CU)
    constexpr int kAhead = SPW > 8 ? 2 : 4;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    f32x4 *red = reinterpret_cast<f32x4 *>(lds);  // [2][kWaves][64]
    char *xl = lds + kSumBytes;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = a.w[0].blocks, steps = blocks >> 2;  // (the same for every layer)
    const int k0 = wave * steps / kWaves, cnt = (wave + 1) * steps / kWaves - k0;

    // the layer, output row and weight of tile t
    int li = 0, row0 = 0;
    u32v4 wv[SPW];
    int ws[SPW];
    auto load_tile = [&](int t) {
        li = 0;
        for (int j = 1; j < a.count; ++j)
            if (t >= a.first[j]) li = j;
        row0 = (t - a.first[li]) * 16;
        const int r = row0 + c;  // n_pad is a multiple of 32: every row of the tile is there
        const uint8_t *wc = a.w[li].codes + ((static_cast<size_t>(r >> 5) * blocks + 4 * k0 + g) * 32 + (r & 31)) * 16;
        const uint8_t *wsc = a.w[li].scales + ((static_cast<size_t>(r >> 5) * steps + k0) * 32 + (r & 31)) * 4 + g;
#pragma unroll
        for (int u = 0; u < SPW; ++u)
            if (u < cnt) {
                wv[u] = *reinterpret_cast<const u32v4 *>(wc + u * 2048);
                ws[u] = wsc[u * 128];
            }
    };
    int t = blockIdx.x;
    load_tile(t);

    using X = XLds<ACT>;
    const int cp = X::code_pitch(blocks), sp = X::scale_pitch(blocks);
    char *xsl = xl + a.batch * cp;
    if constexpr (XT == kBlocks) {
        const int per = X::row_bytes(blocks) / 16, all = a.batch * per;
        for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kThreads) {
            u32v4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (const int i = i0 + j * kThreads; i < all)
                    v[j] = *reinterpret_cast<const u32v4 *>(static_cast<const uint8_t *>(a.x) + static_cast<size_t>(i) * 16);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (const int i = i0 + j * kThreads; i < all) {
                    const int row = i / per, q = i - row * per;
                    *reinterpret_cast<u32v4 *>(xl + row * cp + q * 16) = v[j];
                }
        }
        for (int i = threadIdx.x; i < a.batch * steps; i += kThreads) {
            const int row = i / steps, q = i - row * steps;
            *reinterpret_cast<uint32_t *>(xsl + row * sp + q * 4) = reinterpret_cast<const uint32_t *>(a.xs)[i];
        }
    } else {
        const int m = a.w[0].m, per = blocks * 2, all = a.batch * per;  // units of 16 columns
        mx_saturate(true);
        for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kThreads) {  // (whole pairs of lanes: per is even)
            u32v4 lo[kAhead], hi[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + j * kThreads, row = i / per, col = (i - row * per) * 16;
                const uint16_t *src = static_cast<const uint16_t *>(a.x) + static_cast<size_t>(row) * m + col;
                lo[j] = hi[j] = u32v4{0u, 0u, 0u, 0u};  // columns past m (a multiple of 8) are zeros
                if (i < all && col < m) lo[j] = *reinterpret_cast<const u32v4 *>(src);
                if (i < all && col + 8 < m) hi[j] = *reinterpret_cast<const u32v4 *>(src + 8);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + j * kThreads, row = i / per, q = i - row * per, col = q * 16;
                if (i >= all) break;
                uint32_t mx = float_bits<XT>(absmax(lo[j], hi[j]));
                const uint32_t other = __builtin_amdgcn_mov_dpp(mx, 0xB1, 0xf, 0xf, true);  // the pair's other lane
                mx = mx > other ? mx : other;
                const uint32_t s = mx_scale_byte<ACT>(mx);
                const u32v4 r = codes16<XT, ACT>(lo[j], hi[j], mx_scale_value(s));
                char *dst = xl + row * cp + col / (ACT == DBF_TYPE_E4M3 ? 1 : 2);
                if constexpr (ACT == DBF_TYPE_E4M3) *reinterpret_cast<u32v4 *>(dst) = r;
                else *reinterpret_cast<u32v2 *>(dst) = u32v2{r[0], r[1]};
                if ((q & 1) == 0) xsl[row * sp + (q >> 1)] = static_cast<char>(s);
            }
        }
        mx_saturate(false);
    }
    __syncthreads();

    // operand and scale byte of this lane's row of x (rows past the batch: any, not written)
    const int xrow = min(c, a.batch - 1);
    constexpr int Step = ACT == DBF_TYPE_E4M3 ? 128 : 64;
    const char *xc = xl + xrow * cp + k0 * Step + 16 * g;
    const uint8_t *xs = reinterpret_cast<const uint8_t *>(xsl) + xrow * sp + k0 * 4 + g;

    for (int it = 0; t < a.tiles; ++it) {
        f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        constexpr int FX = ACT == DBF_TYPE_E4M3 ? 0 : 4;
#pragma unroll
        for (int u = 0; u < SPW; ++u)
            if (u < cnt) {
                u32v4 hi = {0u, 0u, 0u, 0u};
                if constexpr (ACT == DBF_TYPE_E4M3) hi = *reinterpret_cast<const u32v4 *>(xc + u * Step + 64);
                const i32x8 op = operand(*reinterpret_cast<const u32v4 *>(xc + u * Step), hi);
                const int sx = xs[u * 4];
                acc[u & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(wv[u], u32v4{0u, 0u, 0u, 0u}), op,
                                                                             acc[u & 1], 4, FX, 0, ws[u], 0, sx);
            }
        const int layer = li, row = row0;
        const int next = t + gridDim.x;
        if (next < a.tiles) load_tile(next);
        f32x4 *sums = red + (it & 1) * (kWaves * 64);
        sums[wave * 64 + lane] = acc[0] + acc[1];
        __syncthreads();  // (the buffer is written again past the next barrier)
        if (wave == (it & (kWaves - 1))) {
            f32x4 s = sums[lane];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) s += sums[v * 64 + lane];
            // result register v of lane (c, g): batch row c, output row 4 g + v
            const int n = a.w[layer].n, col = row + 4 * g;
            typename E::T *dst = static_cast<typename E::T *>(a.y[layer]) + static_cast<size_t>(c) * n + col;
            if (c < a.batch) {
                if (n % 4 == 0) {
                    if (col < n)
                        *reinterpret_cast<u32v2 *>(dst) =
                            u32v2{static_cast<uint32_t>(E::put(s[0])) | static_cast<uint32_t>(E::put(s[1])) << 16,
                                  static_cast<uint32_t>(E::put(s[2])) | static_cast<uint32_t>(E::put(s[3])) << 16};
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (col + v < n) dst[v] = E::put(s[v]);
                }
            }
        }
        t = next;
    }
}

template <int XT, int ACT, typename E, int SPW>
void launch(MxDecodeArgs &a, hipStream_t s) {
    static std::atomic<uint64_t> asked{0};
    a.tiles = 0;
    for (int i = 0; i < a.count; ++i) {
        a.first[i] = a.tiles;
        a.tiles += (a.w[i].n + 15) / 16;
    }
    const size_t bytes = kSumBytes + XLds<ACT>::bytes(a.batch, a.w[0].blocks);
    // One resident wave of workgroups, two per CU where LDS holds both
    // (14336 x 4096, batch 1: 8.7 us, one per CU 10.1).
    const int wgs = bytes <= 80 * 1024 ? 512 : 256;
    const int per = (a.tiles + wgs - 1) / wgs;  // tiles of a workgroup
    auto kernel = mx_decode_kernel<XT, ACT, E, SPW>;
    if (bytes > 65536) allow_lds(kernel, 160 * 1024, asked);
    launch_kernel(kernel, dim3((a.tiles + per - 1) / per), dim3(kThreads), bytes, s, a);
}

template <int XT, int ACT, typename E>
void choose(MxDecodeArgs &a, hipStream_t s) {
    const int spw = (a.w[0].blocks / 4 + kWaves - 1) / kWaves;
    if (spw <= 4) launch<XT, ACT, E, 4>(a, s);
    else if (spw <= 8) launch<XT, ACT, E, 8>(a, s);
    else launch<XT, ACT, E, 16>(a, s);
}

}  // namespace

bool mx_decode_takes(int batch, int m, int act) {
    const int blocks = round_up_int(m, 128) / 32;
    return batch <= kDecodeMaxBatch && m <= 128 * 16 * kWaves &&
           (act == DBF_TYPE_E4M3 ? XLds<DBF_TYPE_E4M3>::bytes(batch, blocks)
                                 : XLds<DBF_TYPE_E2M1>::bytes(batch, blocks)) <= kMaxXBytes;
}

bool mx_decode_quantizes(int batch, int m) { return m % 8 == 0 && static_cast<int64_t>(batch) * m <= 65536; }

int launch_mx_decode(MxDecodeArgs &a, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!mx_decode_takes(a.batch, a.w[0].m, a.act)) return static_cast<int>(hipErrorInvalidValue);
    auto types = [&](auto xt, auto act) {
        constexpr int XT = decltype(xt)::value, ACT = decltype(act)::value;
        if (a.y_type == DBF_TYPE_F16) choose<XT, ACT, F16>(a, s);
        else choose<XT, ACT, BF16>(a, s);
    };
    using E4 = std::integral_constant<int, DBF_TYPE_E4M3>;
    using E2 = std::integral_constant<int, DBF_TYPE_E2M1>;
    auto rows = [&](auto xt) {
        if (a.act == DBF_TYPE_E4M3) types(xt, E4{});
        else types(xt, E2{});
    };
    if (a.x_type == DBF_TYPE_F16) rows(std::integral_constant<int, DBF_TYPE_F16>{});
    else if (a.x_type == DBF_TYPE_BF16) rows(std::integral_constant<int, DBF_TYPE_BF16>{});
    else rows(std::integral_constant<int, kBlocks>{});
    return static_cast<int>(hipGetLastError());
}

}  // namespace dbf
