// Root-mean-square norm with the residual's addition, and its gradient.
//
//   h = rne16(x + r),  rstd = 1 / sqrt(mean(h²) + eps),  y = h rstd w
//   g = dy w,  dx = rstd (g - h rstd² mean(g h)) + dh,  dw = Σ_rows dy h rstd
//
// Every kernel reads a row once and keeps it in registers, eight consecutive
// columns per lane and chunk, so both directions are bound by memory; the
// gradient's next row is on its way while one is reduced and written.  A row's
// squares are formed and added in fp64: a bf16 row's may be far outside of
// fp32, and an error of their mean shifts the whole row at once, which in
// blocks shows as codes on the other side of a tie.  The gradient's sums are
// fp32, over the columns or the rows of a lane.  All joins are in a fixed
// order (no atomics: repeated calls give the same bits).
// y leaves in 16 bits, or in e4m3 blocks of 32 columns with one scale each,
// quantised from the fp32 values: four neighbouring lanes hold a block.
//
// bf16, operands from HBM, graph replays: norm with residual 8192 x 4096
// 56 us (4.8 TB/s moved; squares in fp32 54), with block output 52 us,
// 2048 x 4096 15.2 and 17.9, one row 3.2 and 3.6; gradient with dh 8192 x 4096
// 57 us (4.7 TB/s), 2048 x 4096 22 (a second launch and the parts of dw),
// 65536 x 128 20.

#include <algorithm>

#include "mx_device.h"

namespace dbf {
namespace {

// Sum over the LPR lanes that share a row; every one gets it.  Up to a wave
// without LDS; wider rows meet in red[waves of the workgroup], one barrier.
template <int LPR, typename V>
__device__ __forceinline__ V row_sum(V v, V *red) {
#pragma unroll
    for (int o = (LPR < 64 ? LPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (LPR > 64) {
        const int wave = threadIdx.x >> 6, first = threadIdx.x / LPR * (LPR / 64);
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[first];
#pragma unroll
        for (int i = 1; i < LPR / 64; ++i) v += red[first + i];
    }
    return v;
}

// Eight consecutive 16-bit elements as they are (load8's rules).
template <bool VEC>
__device__ __forceinline__ u32v4 load_raw(const uint16_t *p, int valid) {
    u32v4 q = {0u, 0u, 0u, 0u};
    if constexpr (VEC) {
        if (valid > 0) q = *reinterpret_cast<const u32v4 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) q[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
    return q;
}

template <typename E>
__device__ __forceinline__ void unpack(u32v4 q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = E::get(static_cast<uint16_t>(q[i] & 0xffffu));
        v[2 * i + 1] = E::get(static_cast<uint16_t>(q[i] >> 16));
    }
}

template <typename E, bool VEC>
__device__ __forceinline__ void load_weight(const void *w, int w_f32, int col, int cols, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    } else if (w_f32) {
        load8<F32, VEC>(static_cast<const float *>(w) + col, cols - col, v);
    } else {
        load8<E, VEC>(static_cast<const typename E::T *>(w) + col, cols - col, v);
    }
}

struct NormArgs {
    const void *x, *r, *w;
    int w_f32;
    int rows, cols;
    float eps;
    void *h, *y;
    uint8_t *ys;   // scales of an e4m3 output
    float *rstd;

    // Rows r0 on, `most` of them at most.
    template <typename T, bool MX>
    NormArgs from_row(int64_t r0, int most) const {
        const size_t at = static_cast<size_t>(r0) * cols, wide = (cols + 127) / 128 * 128;
        NormArgs b = *this;
        b.rows = static_cast<int>(std::min<int64_t>(rows - r0, most));
        b.x = static_cast<const T *>(x) + at;
        if (r) b.r = static_cast<const T *>(r) + at;
        if (h) b.h = static_cast<T *>(h) + at;
        if (rstd) b.rstd = rstd + r0;
        if (MX) {
            b.y = static_cast<uint8_t *>(y) + r0 * wide;
            b.ys = ys + r0 * (wide / 32);
        } else {
            b.y = static_cast<T *>(y) + at;
        }
        return b;
    }
};

// LPR lanes per row, NC chunks of 8 LPR columns.
template <typename E, bool MX, bool VEC, int LPR, int NC>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void rms_norm_kernel(const NormArgs a) {
    constexpr int Threads = LPR > 256 ? LPR : 256, RPB = Threads / LPR;
    __shared__ double red[Threads / 64];
    using T = typename E::T;
    const int t = threadIdx.x % LPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LPR;
    if (row >= a.rows) return;  // (RPB > 1 only: no barrier follows)
    const size_t base = static_cast<size_t>(row) * a.cols;
    u32v4 x[NC], r[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * LPR + t) * 8;
        x[c] = load_raw<VEC>(static_cast<const T *>(a.x) + base + col, a.cols - col);
        if (a.r) r[c] = load_raw<VEC>(static_cast<const T *>(a.r) + base + col, a.cols - col);
    }
    float h[NC][8], w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_weight<E, VEC>(a.w, a.w_f32, (c * LPR + t) * 8, a.cols, w[c]);
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * LPR + t) * 8;
        unpack<E>(x[c], h[c]);
        if (a.r) {
            float v[8];
            unpack<E>(r[c], v);
            // the sum of two 16-bit values rounded to fp32 and then to 16
            // bits is their sum rounded once (24 >= 2 * 11 + 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = E::get(E::put(h[c][i] + v[i]));
            if (a.h) store8<E, VEC>(static_cast<T *>(a.h) + base + col, a.cols - col, h[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(h[c][i]), static_cast<double>(h[c][i]), sum);
    }
    sum = row_sum<LPR>(sum, red);
    const double square = sum / a.cols + static_cast<double>(a.eps);
    // 0 where 1 / rms is below fp32's normal numbers: fewer bits than the gradient needs
    double inv = square >= 0x1p252 ? 0.0 : rsqrt(square);
    if (a.rstd && t == 0) a.rstd[row] = static_cast<float>(inv);
    // Rows far from 1 go by a power of two first: no product below leaves
    // fp32's range where the result does not (for weights below 2^104).
    if (!(inv >= 0x1p-16 && inv <= 0x1p16) && inv != 0.0) {
        int ex = 0;
        inv = frexp(inv, &ex);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = ldexpf(h[c][i], ex);
    }
    const float rstd = static_cast<float>(inv), low = static_cast<float>(inv - static_cast<double>(rstd));
    const int wide = (a.cols + 127) / 128 * 128;
    if constexpr (MX) mx_saturate(true);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * LPR + t) * 8;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[c][i] * rstd * w[c][i];
        if constexpr (MX) {
            // Codes show an error of the last fp32 bit where a value is next
            // to the middle of two: one rounding of the product with rstd +
            // low (48 bits), as from 64 bits.  2048 x 4096 17.9 us; three
            // fp32 roundings 17.5, products in fp64 18.7.
            if (!a.w_f32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = h[c][i] * w[c][i];  // exact: 11 or 8 bits each
                    y[i] = fmaf(p, rstd, p * low);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = h[c][i] * rstd;
                    y[i] = fmaf(q, w[c][i], fmaf(h[c][i], low, fmaf(h[c][i], rstd, -q)) * w[c][i]);
                }
            }
        }
        if constexpr (MX) {
            if (col < wide) {
                if (col >= a.cols) {  // padding of the row: zero codes and scales whatever rstd is
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
                } else if (!VEC) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = col + i < a.cols ? y[i] : 0.0f;
                }
                mx_store8<DBF_TYPE_E4M3>(y, col, static_cast<uint8_t *>(a.y) + static_cast<size_t>(row) * wide,
                                         a.ys + static_cast<size_t>(row) * (wide / 32) + (col >> 5));
            }
        } else {
            store8<E, VEC>(static_cast<T *>(a.y) + base + col, a.cols - col, y);
        }
    }
}

struct NormGradArgs {
    const void *dy, *h, *w;
    int w_f32;
    const float *rstd;
    const void *dh;
    int rows, cols;
    void *dx;
    float *part;  // [workgroups][cols] sums of dy h rstd, or null
};

// LPR lanes per row, Threads / LPR rows of a workgroup at a time, gridDim.x
// workgroups in turn.  The sums of dw stay in registers over all rows of a
// lane and are joined in LDS at the end, so a workgroup has one part.
template <typename E, bool VEC, int LPR, int NC, int Threads>
__global__ __launch_bounds__(Threads) void rms_norm_grad_kernel(const NormGradArgs a) {
    constexpr int RPB = Threads / LPR;
    __shared__ float red[2][Threads / 64];  // (in turn: a row's sums are read while the next row's are written)
    __shared__ float joined[RPB > 1 ? RPB / 2 : 1][RPB > 1 ? NC * 8 : 1][RPB > 1 ? LPR : 1];
    using T = typename E::T;
    const int t = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    float dw[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    u32v4 nh[NC], ng[NC], ne[NC];
    float nr = 0.0f;
    auto load_row = [&](int64_t row) {
        if (row >= a.rows) row = a.rows - 1;  // (loaded and not used)
        const size_t base = static_cast<size_t>(row) * a.cols;
        nr = a.rstd[row];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * LPR + t) * 8;
            nh[c] = load_raw<VEC>(static_cast<const T *>(a.h) + base + col, a.cols - col);
            ng[c] = load_raw<VEC>(static_cast<const T *>(a.dy) + base + col, a.cols - col);
            if (a.dh) ne[c] = load_raw<VEC>(static_cast<const T *>(a.dh) + base + col, a.cols - col);
        }
    };
    load_row(static_cast<int64_t>(blockIdx.x) * RPB + sub);
    int turn = 0;
    // (the same number of steps for every row of the workgroup: a barrier may be inside)
    const int64_t stride = static_cast<int64_t>(gridDim.x) * RPB;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * RPB; first < a.rows; first += stride, turn ^= 1) {
        const int64_t row = first + sub;
        const bool here = row < a.rows;
        const size_t base = static_cast<size_t>(row) * a.cols;
        const float rstd = nr;
        float h[NC][8], g[NC][8];
        u32v4 e[NC];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * LPR + t) * 8;
            float w[8];
            unpack<E>(nh[c], h[c]);
            unpack<E>(ng[c], g[c]);
            e[c] = ne[c];
            load_weight<E, VEC>(a.w, a.w_f32, col, a.cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] *= rstd;
                if (here) dw[c][i] += g[c][i] * h[c][i];
                g[c][i] *= w[i];
                sum += g[c][i] * h[c][i];
            }
        }
        // the next row is on its way while this one is finished
        if (first + stride < a.rows) load_row(first + stride + sub);
        sum = row_sum<LPR>(sum, red[turn]);
        const float mean = sum / static_cast<float>(a.cols);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * LPR + t) * 8;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rstd * (g[c][i] - h[c][i] * mean);
            if (a.dh) {
                float v[8];
                unpack<E>(e[c], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += v[i];
            }
            if (a.dx && here) store8<E, VEC>(static_cast<T *>(a.dx) + base + col, a.cols - col, d);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int half = RPB / 2; half > 0; half >>= 1) {
        if (sub >= half && sub < 2 * half) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) joined[sub - half][c * 8 + i][t] = dw[c][i];
        }
        __syncthreads();
        if (sub < half) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[c][i] += joined[sub][c * 8 + i][t];
        }
        __syncthreads();
    }
    if (sub == 0) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * LPR + t) * 8;
            store8<F32, VEC>(a.part + static_cast<size_t>(blockIdx.x) * a.cols + col, a.cols - col, dw[c]);
        }
    }
}

// dw[c] = Σ_p part[p][c]: 64 strips of p, each in order, then eight by eight.
// 16 columns per workgroup, so that 4096 columns use every CU.
__global__ __launch_bounds__(1024) void norm_dw_finish_kernel(const float *__restrict__ part, int parts, int cols,
                                                              float *__restrict__ dw) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, strip = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;
    const int per = (parts + 63) / 64, lo = strip * per, hi = lo + per < parts ? lo + per : parts;
    float v = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int p = lo; p < hi; ++p) v += part[static_cast<size_t>(p) * cols + col];
    }
    s[strip][c] = v;
    __syncthreads();
    if (strip < 8) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += s[strip * 8 + i][c];
    }
    __syncthreads();
    if (strip < 8) s[strip][c] = v;
    __syncthreads();
    if (strip == 0 && col < cols) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += s[i][c];
        dw[col] = v;
    }
}

constexpr int kNormMaxCols = 32768;

// f(lanes per row, chunks per lane) for a width: a lane holds one or two
// chunks of 16 bytes (four from 16384 columns on).  Two of 512 lanes instead
// of four of 256 at 4096 x 8192: gradient 58 instead of 72 us; a
// row of 256 columns on 32 lanes instead of 64 at 65536 rows: 32 instead of 54.
template <int L>
using Int = std::integral_constant<int, L>;
template <typename F>
int by_width(int cols, F f) {
    if (cols <= 128) return f(Int<16>{}, Int<1>{});
    if (cols <= 256) return f(Int<32>{}, Int<1>{});
    if (cols <= 512) return f(Int<64>{}, Int<1>{});
    if (cols <= 1024) return f(Int<64>{}, Int<2>{});
    if (cols <= 2048) return f(Int<256>{}, Int<1>{});
    if (cols <= 4096) return f(Int<256>{}, Int<2>{});
    if (cols <= 8192) return f(Int<512>{}, Int<8192 / 8 / 512>{});
    if (cols <= 16384) return f(Int<1024>{}, Int<16384 / 8 / 1024>{});
    return f(Int<1024>{}, Int<4>{});
}

template <typename E, bool MX>
int launch_norm(const NormArgs &a, hipStream_t s) {
    return by_width(a.cols, [&](auto lpr, auto nc) {
        constexpr int LPR = decltype(lpr)::value, NC = decltype(nc)::value;
        constexpr int Threads = LPR > 256 ? LPR : 256, RPB = Threads / LPR;
        const dim3 block(Threads);
        // A launch holds less than 2^32 threads; more rows are several launches
        // (a loop over rows in the kernel: 8192 x 4096 60 instead of 55 us).
        constexpr int kRows = (1 << 21) * RPB;
        for (int64_t r0 = 0; r0 < a.rows; r0 += kRows) {
            const NormArgs b = a.template from_row<typename E::T, MX>(r0, kRows);
            const dim3 grid(static_cast<uint32_t>((b.rows - 1) / RPB + 1));
            if (a.cols % 8 == 0) launch_kernel(rms_norm_kernel<E, MX, true, LPR, NC>, grid, block, 0, s, b);
            else launch_kernel(rms_norm_kernel<E, MX, false, LPR, NC>, grid, block, 0, s, b);
        }
        return static_cast<int>(hipGetLastError());
    });
}

// Threads of a gradient workgroup: as many rows at a time, and so as few parts
// of dw, as registers allow (two chunks at 1024 threads spill: 8192 x 4096 84
// instead of 57 us; 256 threads and 512 workgroups: 60 us).
constexpr int grad_threads(int lpr, int nc) { return nc == 1 ? 1024 : lpr > 512 ? lpr : 512; }

// Workgroups of the gradient kernel, one per CU, each with its part of dw
// (two per CU at 8192 x 4096: 61 us).
int norm_grad_parts(int rows, int cols) {
    return by_width(cols, [&](auto lpr, auto nc) {
        constexpr int RPB = grad_threads(decltype(lpr)::value, decltype(nc)::value) / decltype(lpr)::value;
        const int need = (rows - 1) / RPB + 1;
        return need < 256 ? need : 256;
    });
}

template <typename E>
int launch_norm_grad(const NormGradArgs &a, hipStream_t s) {
    return by_width(a.cols, [&](auto lpr, auto nc) {
        constexpr int LPR = decltype(lpr)::value, NC = decltype(nc)::value, Threads = grad_threads(LPR, NC);
        const dim3 grid(static_cast<uint32_t>(norm_grad_parts(a.rows, a.cols))), block(Threads);
        if (a.cols % 8 == 0) launch_kernel(rms_norm_grad_kernel<E, true, LPR, NC, Threads>, grid, block, 0, s, a);
        else launch_kernel(rms_norm_grad_kernel<E, false, LPR, NC, Threads>, grid, block, 0, s, a);
        return static_cast<int>(hipGetLastError());
    });
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dbf_status_t check_sizes(int32_t rows, int32_t cols, int32_t type, int32_t weight_type) {
    if (rows < 0 || cols < 1) return DBF_ERR_INVALID_ARG;
    if (type != DBF_TYPE_F16 && type != DBF_TYPE_BF16) return DBF_ERR_INVALID_ARG;
    if (weight_type != type && weight_type != DBF_TYPE_F32) return DBF_ERR_INVALID_ARG;
    if (cols > kNormMaxCols) return DBF_ERR_SHAPE;
    return DBF_OK;
}

}  // namespace
}  // namespace dbf

extern "C" dbf_status_t dbf_rms_norm(const void *x, const void *residual, const void *weight, int32_t type,
                                     int32_t weight_type, int32_t rows, int32_t cols, float eps, void *h, void *y,
                                     int32_t y_type, uint8_t *y_scales, float *rstd, hipStream_t stream) {
    using namespace dbf;
    const dbf_status_t st = check_sizes(rows, cols, type, weight_type);
    if (st != DBF_OK) return st;
    if (!(eps >= 0.0f) || (y_type != type && y_type != DBF_TYPE_E4M3)) return DBF_ERR_INVALID_ARG;
    if (rows == 0) return DBF_OK;
    const bool mx = y_type == DBF_TYPE_E4M3;
    if (!x || !y || (mx && !y_scales) || (!residual && h)) return DBF_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(y) ||
        !aligned4(rstd))
        return DBF_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, weight_type == DBF_TYPE_F32, rows, cols, eps, h, y, y_scales, rstd};
    int e;
    if (type == DBF_TYPE_F16) e = mx ? launch_norm<F16, true>(a, stream) : launch_norm<F16, false>(a, stream);
    else e = mx ? launch_norm<BF16, true>(a, stream) : launch_norm<BF16, false>(a, stream);
    return e == 0 ? DBF_OK : DBF_ERR_HIP;
}

extern "C" size_t dbf_rms_norm_backward_workspace(int32_t rows, int32_t cols) {
    if (rows < 1 || cols < 1) return 0;
    return sizeof(float) * static_cast<size_t>(dbf::norm_grad_parts(rows, cols)) * static_cast<size_t>(cols);
}

extern "C" dbf_status_t dbf_rms_norm_backward(const void *dy, const void *h, const void *weight, const float *rstd,
                                              const void *dh, int32_t type, int32_t weight_type, int32_t rows,
                                              int32_t cols, void *dx, float *dweight, void *workspace,
                                              size_t workspace_bytes, hipStream_t stream) {
    using namespace dbf;
    const dbf_status_t st = check_sizes(rows, cols, type, weight_type);
    if (st != DBF_OK) return st;
    if (rows == 0 && !dweight) return DBF_OK;
    if (dweight && !aligned16(dweight)) return DBF_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!dy || !h || !rstd || !aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned4(rstd) ||
            !aligned16(dh) || !aligned16(dx))
            return DBF_ERR_INVALID_ARG;
        if (dweight && (!workspace || !aligned16(workspace) ||
                        workspace_bytes < dbf_rms_norm_backward_workspace(rows, cols)))
            return DBF_ERR_INVALID_ARG;
        const NormGradArgs a{dy, h, weight, weight_type == DBF_TYPE_F32, rstd, dh, rows, cols, dx,
                             dweight ? static_cast<float *>(workspace) : nullptr};
        const int e = type == DBF_TYPE_F16 ? launch_norm_grad<F16>(a, stream) : launch_norm_grad<BF16>(a, stream);
        if (e != 0) return DBF_ERR_HIP;
    }
    if (dweight) {  // (no rows: zeros)
        launch_kernel(norm_dw_finish_kernel, dim3((cols + 15) / 16), dim3(1024), 0, stream,
                      static_cast<const float *>(workspace), rows > 0 ? norm_grad_parts(rows, cols) : 0, cols, dweight);
        if (hipGetLastError() != hipSuccess) return DBF_ERR_HIP;
    }
    return DBF_OK;
}
