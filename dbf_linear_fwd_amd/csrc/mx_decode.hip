// Products with a 4-bit block weight for few rows (batch 1..64).
//
// The weight's bytes are all there is to move, so the kernel streams them
// once: a workgroup takes 16 or 32 output rows, its waves cut K between them,
// and each wave multiplies 16 weight rows x 128 columns with 16 rows of x per
// matrix-core instruction (the weight as the first operand, the batch as the
// second one's columns; a batch of one costs the same as 16).  The waves'
// sums meet in LDS and are added in wave order.
//
// Of the 16x16x128 instruction a lane (c = lane % 16, g = lane / 16) supplies
// row c: of an e2m1 operand the 16 bytes of block g; of an e4m3 operand bytes
// 16 g .. of the first 64 columns and of the second 64.  Its scale byte is
// block g's either way.
//
// f16 and bf16 rows up to batch 16 are quantised in registers, with no pass
// or launch of their own: an e2m1 lane holds a whole block, an e4m3 lane
// halves of two blocks, which two lane-group swaps bring together.  Every
// workgroup quantises the x that it reads; at 16 rows this is about 60
// instructions per KiB of weight, hidden behind its loads.

#include "mx_device.h"

namespace dbf {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Rows of x as the kernel's template argument: 16-bit values, or ready blocks.
constexpr int kBlocks = -1;

__device__ __forceinline__ i32x8 operand(u32v4 a, u32v4 b) {
    return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                 static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}

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

template <int XT, int ACT>
__device__ __forceinline__ u32v4 codes16(u32v4 a, u32v4 b, float sc) {
    // 16 values: e4m3 in four words; e2m1 in two (words 0, 1)
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

// The operand words and the scale byte of this lane from its 32 16-bit
// values v[0..3] (eight each).  FP16_OVFL must be on (e4m3 saturates).
template <int XT, int ACT>
__device__ __forceinline__ void quantize_lane(const u32v4 (&v)[4], i32x8 &op, int &scale) {
    const u32v4 z = {0u, 0u, 0u, 0u};
    if constexpr (ACT == DBF_TYPE_E2M1) {
        const uint32_t m = max16x2(absmax(v[0], v[1]), absmax(v[2], v[3]));
        const uint32_t s = mx_scale_byte<ACT>(float_bits<XT>(m));
        const float sc = mx_scale_value(s);
        const u32v4 a = codes16<XT, ACT>(v[0], v[1], sc), b = codes16<XT, ACT>(v[2], v[3], sc);
        op = operand(u32v4{a[0], a[1], b[0], b[1]}, z);
        scale = static_cast<int>(s);
    } else {
        // lane group g holds half g % 2 of blocks g / 2 and 2 + g / 2.  The
        // swap exchanges odd lane groups of its first value with even ones of
        // its second: the two halves of block 0, 2, 1, 3 meet in groups 0..3.
        const uint32_t m0 = float_bits<XT>(absmax(v[0], v[1])), m1 = float_bits<XT>(absmax(v[2], v[3]));
        const auto p = __builtin_amdgcn_permlane16_swap(m0, m1, false, false);
        const uint32_t pa = p[0], pb = p[1];
        const uint32_t s = mx_scale_byte<ACT>(pa > pb ? pa : pb);  // of block 0, 2, 1, 3 in groups 0..3
        const auto q = __builtin_amdgcn_permlane16_swap(s, s, false, false);
        const uint32_t s0 = q[0], s1 = q[1];  // of blocks g / 2 and 2 + g / 2
        const u32v4 a = codes16<XT, ACT>(v[0], v[1], mx_scale_value(s0));
        const u32v4 b = codes16<XT, ACT>(v[2], v[3], mx_scale_value(s1));
        op = operand(a, b);
        const auto h = __builtin_amdgcn_permlane32_swap(s0, s1, false, false);  // blocks 0 0 2 2 and 1 1 3 3
        const uint32_t h0 = h[0], h1 = h[1];
        const auto t = __builtin_amdgcn_permlane16_swap(h0, h1, false, false);  // 0 1 2 3
        const uint32_t t0 = t[0];
        scale = static_cast<int>(t0);
    }
}

// XT: type of x's rows (f16, bf16) or kBlocks; RT: 16-row weight tiles per
// workgroup; NB: groups of 16 rows of x; U: steps of 128 columns in flight.
template <int XT, int ACT, typename E, int RT, int NB, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void mx_decode_kernel(const MxDecodeArgs a) {
    __shared__ __attribute__((aligned(16))) f32x4 red[WAVES][RT * NB][64];
    int li = 0;
    for (int j = 1; j < a.count; ++j)
        if (static_cast<int>(blockIdx.x) >= a.first[j]) li = j;
    const MxWeight &w = a.w[li];
    const int row0 = (static_cast<int>(blockIdx.x) - a.first[li]) * 16 * RT;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = w.blocks, steps = blocks >> 2;
    const int k0 = wave * steps / WAVES, k1 = (wave + 1) * steps / WAVES;

    const uint8_t *wc[RT], *ws[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = row0 + 16 * t + c;  // n_pad is a multiple of 32: every row of the tile is there
        wc[t] = w.codes + ((static_cast<size_t>(r >> 5) * blocks + g) * 32 + (r & 31)) * 16;
        ws[t] = w.scales + (static_cast<size_t>(r >> 5) * steps * 32 + (r & 31)) * 4 + g;
    }
    const uint8_t *xr[NB], *xsr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int row = min(16 * b + c, a.batch - 1);  // rows past the batch: multiplied, not written
        if constexpr (XT == kBlocks) {
            xr[b] = static_cast<const uint8_t *>(a.x) + static_cast<size_t>(row) * blocks * (ACT == DBF_TYPE_E4M3 ? 32 : 16) + 16 * g;
            xsr[b] = a.xs + static_cast<size_t>(row) * blocks + g;
        } else {
            xr[b] = static_cast<const uint8_t *>(a.x) + (static_cast<size_t>(row) * w.m + (ACT == DBF_TYPE_E4M3 ? 16 : 32) * g) * 2;
            xsr[b] = nullptr;
        }
    }
    f32x4 acc[RT][NB];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (XT != kBlocks) mx_saturate(true);

    for (int k = k0; k < k1; k += U) {
        u32v4 wv[U][RT], xv[U][NB][XT == kBlocks ? 2 : 4];
        int wsc[U][RT], xsc[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kt = min(k + u, k1 - 1);  // (past the end: loaded, not multiplied)
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                wv[u][t] = *reinterpret_cast<const u32v4 *>(wc[t] + static_cast<size_t>(kt) * 2048);
                wsc[u][t] = ws[t][static_cast<size_t>(kt) * 128];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kt = min(k + u, k1 - 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (XT == kBlocks) {
                    if constexpr (ACT == DBF_TYPE_E4M3) {
                        xv[u][b][0] = *reinterpret_cast<const u32v4 *>(xr[b] + static_cast<size_t>(kt) * 128);
                        xv[u][b][1] = *reinterpret_cast<const u32v4 *>(xr[b] + static_cast<size_t>(kt) * 128 + 64);
                    } else {
                        xv[u][b][0] = *reinterpret_cast<const u32v4 *>(xr[b] + static_cast<size_t>(kt) * 64);
                        xv[u][b][1] = u32v4{0u, 0u, 0u, 0u};
                    }
                    xsc[u][b] = xsr[b][static_cast<size_t>(kt) * 4];
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // eight values; columns past m (a multiple of 8) are zeros
                        const int off = ACT == DBF_TYPE_E4M3 ? 64 * (q >> 1) + 8 * (q & 1) : 8 * q;
                        const int col = kt * 128 + (ACT == DBF_TYPE_E4M3 ? 16 : 32) * g + off;
                        xv[u][b][q] = u32v4{0u, 0u, 0u, 0u};
                        if (col < w.m) xv[u][b][q] = *reinterpret_cast<const u32v4 *>(xr[b] + (static_cast<size_t>(kt) * 128 + off) * 2);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u >= k1) break;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                i32x8 op;
                int sx;
                if constexpr (XT == kBlocks) {
                    op = operand(xv[u][b][0], xv[u][b][1]);
                    sx = xsc[u][b];
                } else {
                    quantize_lane<XT, ACT>(xv[u][b], op, sx);
                }
                constexpr int FX = ACT == DBF_TYPE_E4M3 ? 0 : 4;
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        operand(wv[u][t], u32v4{0u, 0u, 0u, 0u}), op, acc[t][b], 4, FX, 0, wsc[u][t], 0, sx);
            }
        }
    }
    if constexpr (XT != kBlocks) mx_saturate(false);

#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[wave][t * NB + b][lane] = acc[t][b];
    __syncthreads();
    // result register v of lane (c, g): batch row c, output row 4 g + v
    typename E::T *y = static_cast<typename E::T *>(a.y[li]);
    for (int i = threadIdx.x; i < RT * NB * 64; i += 64 * WAVES) {
        const int f = i >> 6, l = i & 63;
        f32x4 s = red[0][f][l];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) s += red[v][f][l];
        const int row = (f % NB) * 16 + (l & 15), col = row0 + (f / NB) * 16 + 4 * (l >> 4);
        if (row >= a.batch) continue;
        typename E::T *dst = y + static_cast<size_t>(row) * w.n + col;
        if (w.n % 4 == 0) {
            if (col < w.n)
                *reinterpret_cast<u32v2 *>(dst) = u32v2{static_cast<uint32_t>(E::put(s[0])) | static_cast<uint32_t>(E::put(s[1])) << 16,
                                                        static_cast<uint32_t>(E::put(s[2])) | static_cast<uint32_t>(E::put(s[3])) << 16};
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (col + v < w.n) dst[v] = E::put(s[v]);
        }
    }
}

template <int XT, int ACT, typename E, int RT, int NB, int WAVES, int U>
void launch(MxDecodeArgs &a, hipStream_t s) {
    int n = 0;
    for (int i = 0; i < a.count; ++i) {
        a.first[i] = n;
        n += (a.w[i].n + 16 * RT - 1) / (16 * RT);
    }
    launch_kernel(mx_decode_kernel<XT, ACT, E, RT, NB, WAVES, U>, dim3(n), dim3(64 * WAVES), 0, s, a);
}

template <int XT, int ACT, typename E>
void choose(MxDecodeArgs &a, hipStream_t s) {
    if constexpr (XT == kBlocks) {
        if (a.batch > 32) return launch<XT, ACT, E, 1, 4, 8, 2>(a, s);
        if (a.batch > 16) return launch<XT, ACT, E, 1, 2, 8, 4>(a, s);
    }
    launch<XT, ACT, E, 1, 1, 8, 4>(a, s);
}

}  // namespace

int launch_mx_decode(MxDecodeArgs &a, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
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
