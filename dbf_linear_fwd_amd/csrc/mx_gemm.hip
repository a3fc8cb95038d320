// Products with a 4-bit weight in blocks of 32 with power-of-two scales
// (include/dbf.h, "Block formats") on the scaled matrix-core instructions:
//   Y[b][o]  = Σ_l xq[b][l] wq[o][l]      x in e4m3 or e2m1 blocks
//   dX[b][l] = Σ_o dy[b][o] wq[o][l]      dy in f16 or bf16
//
// The 32x32x64 instruction multiplies 64 columns of K per step and applies
// both operands' block scales itself.  A lane (r = lane % 32, g = lane / 32)
// supplies row r: of an e2m1 operand the 16 bytes of block g, of an e4m3
// operand bytes 16g..16g+15 of block 0 and of block 1; its scale byte is
// always that of block g.

#include "mx_device.h"

namespace dbf {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 operand(u32v4 a, u32v4 b) {
    return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                 static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}

// One wave per 32 x 32 output tile.
template <int FMT, typename E>
__global__ __launch_bounds__(256) void mx_product_kernel(const uint8_t *__restrict__ xc,
                                                         const uint8_t *__restrict__ xs, int M, MxWeight w,
                                                         typename E::T *__restrict__ y) {
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
    const int nt = w.n_pad / 32;
    const int64_t tile = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int64_t mt64 = tile / nt;
    if (mt64 * 32 >= M) return;
    const int mt = static_cast<int>(mt64), t = static_cast<int>(tile - mt64 * nt);
    const int row = mt * 32 + r < M ? mt * 32 + r : M - 1;  // rows past M: multiplied, not written
    const int kb = w.blocks;
    constexpr int kBytes = FMT == DBF_TYPE_E4M3 ? 32 : 16;  // of a block
    const uint8_t *xr = xc + static_cast<size_t>(row) * kb * kBytes;
    const uint8_t *xsr = xs + static_cast<size_t>(row) * kb;
    const uint8_t *wt = w.codes + (static_cast<size_t>(t) * kb * 32 + r) * 16;
    const uint8_t *wst = w.scales + (static_cast<size_t>(t) * (kb >> 2) * 32 + r) * 4;
    f32x16 acc = {};
    for (int b = 0; b < kb; b += 2) {
        u32v4 a0, a1 = {0u, 0u, 0u, 0u};
        if constexpr (FMT == DBF_TYPE_E4M3) {
            a0 = *reinterpret_cast<const u32v4 *>(xr + b * 32 + 16 * g);
            a1 = *reinterpret_cast<const u32v4 *>(xr + b * 32 + 32 + 16 * g);
        } else {
            a0 = *reinterpret_cast<const u32v4 *>(xr + (b + g) * 16);
        }
        const u32v4 z = {0u, 0u, 0u, 0u};
        const u32v4 c = *reinterpret_cast<const u32v4 *>(wt + static_cast<size_t>(b + g) * 512);
        const int sx = xsr[b + g];
        const int sw = wst[static_cast<size_t>((b + g) >> 2) * 128 + ((b + g) & 3)];
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a0, a1), operand(c, z), acc,
                                                              FMT == DBF_TYPE_E4M3 ? 0 : 4, 4, 0, sx, 0, sw);
    }
    const int col = t * 32 + r;
    if (col >= w.n) return;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int o = mt * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
        if (o < M) y[static_cast<size_t>(o) * w.n + col] = E::put(acc[v]);
    }
}

// One wave per 32 rows x 32 columns (one block) of dX.  The weight's values
// enter as code * 2^(s - smax + 13) with smax the largest scale of the block
// column, so that they are exact in f16 unless 2^-37 or less of the largest
// one; the sum is multiplied by 2^(smax - 13) at the end.
template <typename E>
__global__ __launch_bounds__(256) void mx_backward_kernel(const typename E::T *__restrict__ dy, int M, MxWeight w,
                                                          typename E::T *__restrict__ dx) {
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
    const int nb = (w.m + 31) / 32;
    const int64_t tile = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int64_t mt64 = tile / nb;
    if (mt64 * 32 >= M) return;
    const int mt = static_cast<int>(mt64), kb = static_cast<int>(tile - mt64 * nb);
    const int row = mt * 32 + r < M ? mt * 32 + r : M - 1;
    const typename E::T *dyr = dy + static_cast<size_t>(row) * w.n;
    const int smax = w.colmax[kb];
    f32x16 acc = {};
    for (int o0 = 0; o0 < w.n; o0 += 16) {
        uint16_t a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int o = o0 + 8 * g + i, t = o >> 5;
            const bool in = o < w.n;  // (n_pad is a multiple of 32: the weight's rows exist)
            a[i] = in ? dyr[o] : 0;
            const size_t at = (static_cast<size_t>(t) * w.blocks + kb) * 32 + (o & 31);
            const uint32_t byte = w.codes[at * 16 + r / 2];
            const int s = w.scales[((static_cast<size_t>(t) * (w.blocks >> 2) + (kb >> 2)) * 32 + (o & 31)) * 4 + (kb & 3)];
            const int e = s - smax + 13 + 127;
            const float sc = s == 255 ? __builtin_bit_cast(float, 0x7fc00000u)
                                      : __builtin_bit_cast(float, static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
            uint32_t p;
            if constexpr (E::code == DBF_TYPE_BF16)
                p = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(byte, sc, 0));
            else
                p = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(byte, sc, 0));
            b[i] = static_cast<uint16_t>(r & 1 ? p >> 16 : p & 0xffffu);
        }
        if constexpr (E::code == DBF_TYPE_BF16)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<bf16x8 *>(a), *reinterpret_cast<bf16x8 *>(b), acc, 0, 0, 0);
        else
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<f16x8 *>(a), *reinterpret_cast<f16x8 *>(b), acc, 0, 0, 0);
    }
    const int col = kb * 32 + r;
    if (col >= w.m) return;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int o = mt * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
        if (o < M) dx[static_cast<size_t>(o) * w.m + col] = E::put(ldexpf(acc[v], smax - 127 - 13));
    }
}

}  // namespace

int launch_mx_product(const MxProduct &p, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t tiles = static_cast<int64_t>((p.M + 31) / 32) * (p.w.n_pad / 32);
    const dim3 grid(static_cast<uint32_t>((tiles + 3) / 4));
    auto go = [&](auto f, auto e) {
        using E = decltype(e);
        launch_kernel(mx_product_kernel<decltype(f)::value, E>, grid, dim3(256), 0, s,
                      static_cast<const uint8_t *>(p.xcodes), p.xscales, p.M, p.w, static_cast<typename E::T *>(p.y));
    };
    auto pick = [&](auto f) {
        if (p.y_type == DBF_TYPE_F16) go(f, F16{});
        else if (p.y_type == DBF_TYPE_BF16) go(f, BF16{});
        else go(f, F32{});
    };
    if (p.x_type == DBF_TYPE_E4M3) pick(std::integral_constant<int, DBF_TYPE_E4M3>{});
    else pick(std::integral_constant<int, DBF_TYPE_E2M1>{});
    return static_cast<int>(hipGetLastError());
}

int launch_mx_backward(const void *dy, int type, int M, const MxWeight &w, void *dx, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t tiles = static_cast<int64_t>((M + 31) / 32) * ((w.m + 31) / 32);
    const dim3 grid(static_cast<uint32_t>((tiles + 3) / 4));
    if (type == DBF_TYPE_BF16)
        launch_kernel(mx_backward_kernel<BF16>, grid, dim3(256), 0, s, static_cast<const uint16_t *>(dy), M, w, static_cast<uint16_t *>(dx));
    else
        launch_kernel(mx_backward_kernel<F16>, grid, dim3(256), 0, s, static_cast<const uint16_t *>(dy), M, w, static_cast<uint16_t *>(dx));
    return static_cast<int>(hipGetLastError());
}

}  // namespace dbf
