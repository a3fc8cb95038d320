// Quantisation to and from the block formats, and the device layout of a
// 4-bit weight.
//
// A block of 32 columns with largest magnitude amax takes the scale
// 2^(floor(log2 amax) - E) (E = 8 for e4m3, 2 for e2m1), so its values lie in
// [0, 2^(E+1)) and the top of that range saturates at 448 / 6; each value is
// rounded once, to nearest even, by the conversion instruction.  All of it
// is bound by memory: 2 or 4 bytes read and 1/2 or 1 (+ 1/32) written per
// value.

#include "mx_device.h"

namespace dbf {
namespace {

// One lane per eight columns, four neighbouring lanes per block: 16 bytes
// (32 of fp32) read and 8 or 4 written by each lane, contiguous over the wave.
template <typename E, int FMT, bool VEC>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const typename E::T *__restrict__ x, uint32_t rows,
                                                          int cols, int wide, uint8_t *__restrict__ codes,
                                                          uint8_t *__restrict__ scales, int tiled) {
    const uint32_t per_row = static_cast<uint32_t>(wide) / 8;
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = idx / per_row;
    if (row >= rows) return;  // per_row is a multiple of 16: whole blocks leave together
    const int col = static_cast<int>(idx - row * per_row) * 8;
    float v[8];
    load8<E, VEC>(x + static_cast<size_t>(row) * cols + col, cols - col, v);
    constexpr int kPer = FMT == DBF_TYPE_E4M3 ? 1 : 2;  // columns per byte
    if constexpr (FMT == DBF_TYPE_E4M3) mx_saturate(true);
    // tiled: four scale bytes of a row, then the next row of the 32-row tile
    const int kb = col >> 5;
    uint8_t *at = tiled ? scales + (static_cast<size_t>(row >> 5) * (wide / 128) + (kb >> 2)) * 128 + (row & 31) * 4 + (kb & 3)
                        : scales + static_cast<size_t>(row) * (wide / 32) + kb;
    mx_store8<FMT>(v, col, codes + static_cast<size_t>(row) * (wide / kPer), at);
}

// Values of eight columns per lane.  The conversion instructions multiply by
// the scale and round once (f16, bf16); fp32 takes the code's exact value
// times the scale.
template <typename E, int FMT, bool VEC>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, uint32_t rows,
                                                            int cols, int wide, typename E::T *__restrict__ out) {
    const uint32_t per_row = (static_cast<uint32_t>(cols) + 7) / 8;
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = idx / per_row;
    if (row >= rows) return;
    const int col = static_cast<int>(idx - row * per_row) * 8;
    const float sc = mx_scale_value(scales[static_cast<size_t>(row) * (wide / 32) + (col >> 5)]);
    uint32_t w[2] = {0, 0};
    if constexpr (FMT == DBF_TYPE_E4M3) {
        const u32v2 q = *reinterpret_cast<const u32v2 *>(codes + static_cast<size_t>(row) * wide + col);
        w[0] = q[0];
        w[1] = q[1];
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(codes + static_cast<size_t>(row) * (wide / 2) + col / 2);
    }
    uint32_t pair[4];  // 16-bit results, two per word (fp32: the codes' values in f16, exact)
    auto cvt = [&](auto half, float s) {
        constexpr bool B = decltype(half)::value;
        if constexpr (FMT == DBF_TYPE_E4M3) {
            if constexpr (B) {
                pair[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, false));
                pair[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, true));
                pair[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, false));
                pair[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, true));
            } else {
                pair[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], s, false));
                pair[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], s, true));
                pair[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], s, false));
                pair[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], s, true));
            }
        } else {
            if constexpr (B) {
                pair[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 0));
                pair[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 1));
                pair[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 2));
                pair[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 3));
            } else {
                pair[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], s, 0));
                pair[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], s, 1));
                pair[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], s, 2));
                pair[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], s, 3));
            }
        }
    };
    typename E::T *dst = out + static_cast<size_t>(row) * cols + col;
    const int valid = cols - col;
    if constexpr (E::code == DBF_TYPE_F32) {
        cvt(std::false_type{}, 1.0f);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = F16::get(static_cast<uint16_t>(i & 1 ? pair[i >> 1] >> 16 : pair[i >> 1] & 0xffffu)) * sc;
        store8<E, VEC>(dst, valid, v);
    } else {
        cvt(std::integral_constant<bool, E::code == DBF_TYPE_BF16>{}, sc);
        if constexpr (VEC) {
            *reinterpret_cast<u32v4 *>(dst) = u32v4{pair[0], pair[1], pair[2], pair[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) dst[i] = static_cast<uint16_t>(i & 1 ? pair[i >> 1] >> 16 : pair[i >> 1] & 0xffffu);
        }
    }
}

// Device layout of an e2m1 weight (see MxWeight): one thread per 16-byte
// block of codes; rows n..n_pad-1 are zero.
__global__ __launch_bounds__(256) void mx_layout_kernel(const uint8_t *__restrict__ codes,
                                                        const uint8_t *__restrict__ scales, int n, int n_pad,
                                                        int blocks, uint8_t *__restrict__ out_codes,
                                                        uint8_t *__restrict__ out_scales) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (idx >= static_cast<int64_t>(n_pad) * blocks) return;
    const int r = static_cast<int>(idx & 31);
    const int64_t q = idx >> 5;
    const int kb = static_cast<int>(q % blocks), tile = static_cast<int>(q / blocks);
    const int row = tile * 32 + r;
    u32v4 c = {0u, 0u, 0u, 0u};
    uint8_t s = 0;
    if (row < n) {
        c = *reinterpret_cast<const u32v4 *>(codes + (static_cast<int64_t>(row) * blocks + kb) * 16);
        s = scales[static_cast<int64_t>(row) * blocks + kb];
    }
    *reinterpret_cast<u32v4 *>(out_codes + idx * 16) = c;
    out_scales[((static_cast<int64_t>(tile) * (blocks >> 2) + (kb >> 2)) * 32 + r) * 4 + (kb & 3)] = s;
}

// Largest scale byte (NaN bytes aside) of each block of columns over all rows,
// and 16 zero bytes after the last (what the gradient reads past a row's end).
__global__ __launch_bounds__(256) void mx_colmax_kernel(const uint8_t *__restrict__ scales, int n, int blocks,
                                                        uint8_t *__restrict__ out) {
    const int kb = blockIdx.x;
    int best = 0;
    for (int r = threadIdx.x; r < n; r += 256) {
        const int s = scales[static_cast<int64_t>(r) * blocks + kb];
        if (s != 255 && s > best) best = s;
    }
    __shared__ int red[256];
    red[threadIdx.x] = best;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o && red[threadIdx.x + o] > red[threadIdx.x]) red[threadIdx.x] = red[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[kb] = static_cast<uint8_t>(red[0]);
    if (kb == 0 && threadIdx.x < 16) out[blocks + threadIdx.x] = 0;
}

uint32_t grid_for(uint64_t threads) { return static_cast<uint32_t>((threads + 255) / 256); }

}  // namespace

int launch_mx_quantize(const void *x, int x_type, int rows, int cols, int fmt, void *codes, uint8_t *scales,
                       bool tiled, void *stream) {
    const int wide = round_up_int(cols, 128);
    const dim3 grid(grid_for(static_cast<uint64_t>(rows) * (wide / 8)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool vec = cols % 8 == 0;
    auto go = [&](auto e, auto f) {
        using E = decltype(e);
        constexpr int FMT = decltype(f)::value;
        const auto *p = static_cast<const typename E::T *>(x);
        auto *c = static_cast<uint8_t *>(codes);
        if (vec) launch_kernel(mx_quantize_kernel<E, FMT, true>, grid, dim3(256), 0, s, p, uint32_t(rows), cols, wide, c, scales, int(tiled));
        else launch_kernel(mx_quantize_kernel<E, FMT, false>, grid, dim3(256), 0, s, p, uint32_t(rows), cols, wide, c, scales, int(tiled));
    };
    auto pick = [&](auto f) {
        if (x_type == DBF_TYPE_F16) go(F16{}, f);
        else if (x_type == DBF_TYPE_BF16) go(BF16{}, f);
        else go(F32{}, f);
    };
    if (fmt == DBF_TYPE_E4M3) pick(std::integral_constant<int, DBF_TYPE_E4M3>{});
    else pick(std::integral_constant<int, DBF_TYPE_E2M1>{});
    return static_cast<int>(hipGetLastError());
}

int launch_mx_dequantize(const void *codes, const uint8_t *scales, int fmt, int rows, int cols, void *out,
                         int out_type, void *stream) {
    const int wide = round_up_int(cols, 128);
    const dim3 grid(grid_for(static_cast<uint64_t>(rows) * ((cols + 7) / 8)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool vec = cols % 8 == 0;
    auto go = [&](auto e, auto f) {
        using E = decltype(e);
        constexpr int FMT = decltype(f)::value;
        auto *p = static_cast<typename E::T *>(out);
        const auto *c = static_cast<const uint8_t *>(codes);
        if (vec) launch_kernel(mx_dequantize_kernel<E, FMT, true>, grid, dim3(256), 0, s, c, scales, uint32_t(rows), cols, wide, p);
        else launch_kernel(mx_dequantize_kernel<E, FMT, false>, grid, dim3(256), 0, s, c, scales, uint32_t(rows), cols, wide, p);
    };
    auto pick = [&](auto f) {
        if (out_type == DBF_TYPE_F16) go(F16{}, f);
        else if (out_type == DBF_TYPE_BF16) go(BF16{}, f);
        else go(F32{}, f);
    };
    if (fmt == DBF_TYPE_E4M3) pick(std::integral_constant<int, DBF_TYPE_E4M3>{});
    else pick(std::integral_constant<int, DBF_TYPE_E2M1>{});
    return static_cast<int>(hipGetLastError());
}

int launch_mx_layout(const void *codes, const uint8_t *scales, int n, int m, uint8_t *out_codes, uint8_t *out_scales,
                     uint8_t *colmax, void *stream) {
    const int blocks = round_up_int(m, 128) / 32, n_pad = round_up_int(n, 32);
    hipStream_t s = static_cast<hipStream_t>(stream);
    launch_kernel(mx_layout_kernel, dim3(grid_for(static_cast<uint64_t>(n_pad) * blocks)), dim3(256), 0, s,
                  static_cast<const uint8_t *>(codes), scales, n, n_pad, blocks, out_codes, out_scales);
    launch_kernel(mx_colmax_kernel, dim3(blocks), dim3(256), 0, s, scales, n, blocks, colmax);
    return static_cast<int>(hipGetLastError());
}

}  // namespace dbf

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool is_real(int32_t t) { return t == DBF_TYPE_F16 || t == DBF_TYPE_BF16 || t == DBF_TYPE_F32; }
bool is_block(int32_t t) { return t == DBF_TYPE_E4M3 || t == DBF_TYPE_E2M1; }

dbf_status_t check(const void *x, int32_t x_type, int32_t rows, int32_t cols, int32_t type, const void *codes,
                   const uint8_t *scales) {
    if (rows < 0 || cols < 1 || !is_real(x_type) || !is_block(type)) return DBF_ERR_INVALID_ARG;
    // (one thread per eight columns, counted in 32 bits)
    if (cols > (1 << 30) || static_cast<int64_t>(rows) * dbf::round_up_int(cols, 128) > (int64_t(1) << 34))
        return DBF_ERR_SHAPE;
    if (rows == 0) return DBF_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned4(scales))
        return DBF_ERR_INVALID_ARG;
    return DBF_OK;
}

}  // namespace

extern "C" size_t dbf_mx_code_bytes(int32_t cols, int32_t type) {
    if (cols < 1 || cols > (1 << 30) || !is_block(type)) return 0;
    const size_t wide = static_cast<size_t>(dbf::round_up_int(cols, 128));
    return type == DBF_TYPE_E4M3 ? wide : wide / 2;
}

extern "C" size_t dbf_mx_scale_bytes(int32_t cols) {
    if (cols < 1 || cols > (1 << 30)) return 0;
    return static_cast<size_t>(dbf::round_up_int(cols, 128)) / 32;
}

extern "C" dbf_status_t dbf_mx_quantize(const void *x, int32_t x_type, int32_t rows, int32_t cols, int32_t type,
                                        void *codes, uint8_t *scales, hipStream_t stream) {
    const dbf_status_t st = check(x, x_type, rows, cols, type, codes, scales);
    if (st != DBF_OK || rows == 0) return st;
    return dbf::launch_mx_quantize(x, x_type, rows, cols, type, codes, scales, false, stream) == 0 ? DBF_OK : DBF_ERR_HIP;
}

extern "C" dbf_status_t dbf_mx_dequantize(const void *codes, const uint8_t *scales, int32_t type, int32_t rows,
                                          int32_t cols, void *out, int32_t out_type, hipStream_t stream) {
    const dbf_status_t st = check(out, out_type, rows, cols, type, codes, scales);
    if (st != DBF_OK || rows == 0) return st;
    return dbf::launch_mx_dequantize(codes, scales, type, rows, cols, out, out_type, stream) == 0 ? DBF_OK
                                                                                                 : DBF_ERR_HIP;
}
