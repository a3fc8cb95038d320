// Root-mean-square norm with the residual's addition, and its gradient.
//
//   h = rne16(x + r),  rstd = 1 / sqrt(mean(h²) + eps),  y = h rstd w
//   g = dy w,  dx = rstd (g - h rstd² mean(g h)) + dh,  dw = Σ_rows dy h rstd
//
// Every kernel reads a row once and keeps it in registers, eight consecutive
// columns per lane and chunk, so both directions are bound by memory.  Sums
// are fp32: a lane's own columns in order, then over the wave, then over the
// waves in order (no atomics: repeated calls give the same bits).  y leaves
// in 16 bits, or in e4m3 blocks of 32 columns with one scale each, quantised
// from the fp32 values: four neighbouring lanes hold a block.

#include "mx_device.h"

namespace dbf {
namespace {

// Sum over the wave; every lane gets it.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over the WPR waves that share a row (WPR = 1: no LDS, no barrier).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) v += red[i];
    }
    return v;
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
};

// WPR waves per row (4 / WPR rows per workgroup, at least one), NC chunks of
// 512 * WPR columns.
template <typename E, bool MX, bool VEC, int WPR, int NC>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void rms_norm_kernel(const NormArgs a) {
    constexpr int RPB = WPR >= 4 ? 1 : 4 / WPR;
    __shared__ float red[WPR];
    using T = typename E::T;
    const int t = WPR >= 4 ? threadIdx.x : threadIdx.x % (64 * WPR);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + (WPR >= 4 ? 0 : threadIdx.x / (64 * WPR));
    if (row >= a.rows) return;  // (WPR = 1 only: no barrier follows)
    const size_t base = static_cast<size_t>(row) * a.cols;
    float h[NC][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * 64 * WPR + t) * 8;
        load8<E, VEC>(static_cast<const T *>(a.x) + base + col, a.cols - col, h[c]);
        if (a.r) {
            float r[8];
            load8<E, VEC>(static_cast<const T *>(a.r) + base + col, a.cols - col, r);
            // the sum of two 16-bit values rounded to fp32 and then to 16
            // bits is their sum rounded once (24 >= 2 * 11 + 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = E::get(E::put(h[c][i] + r[i]));
            if (a.h) store8<E, VEC>(static_cast<T *>(a.h) + base + col, a.cols - col, h[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += h[c][i] * h[c][i];
    }
    sum = row_sum<WPR>(sum, red);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    const int wide = (a.cols + 127) / 128 * 128;
    if constexpr (MX) mx_saturate(true);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * 64 * WPR + t) * 8;
        float w[8], y[8];
        load_weight<E, VEC>(a.w, a.w_f32, col, a.cols, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[c][i] * rstd * w[i];
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

// Each workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps
// its sums of dw in registers.
template <typename E, bool VEC, int WPR, int NC>
__global__ __launch_bounds__(64 * WPR) void rms_norm_grad_kernel(const NormGradArgs a) {
    __shared__ float red[WPR];
    using T = typename E::T;
    const int t = threadIdx.x;
    float dw[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * a.cols;
        const float rstd = a.rstd[row];
        float h[NC][8], g[NC][8];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * 64 * WPR + t) * 8;
            float w[8];
            load8<E, VEC>(static_cast<const T *>(a.h) + base + col, a.cols - col, h[c]);
            load8<E, VEC>(static_cast<const T *>(a.dy) + base + col, a.cols - col, g[c]);
            load_weight<E, VEC>(a.w, a.w_f32, col, a.cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] *= rstd;
                dw[c][i] += g[c][i] * h[c][i];
                g[c][i] *= w[i];
                sum += g[c][i] * h[c][i];
            }
        }
        sum = row_sum<WPR>(sum, red);
        if constexpr (WPR > 1) __syncthreads();  // red is free again
        const float mean = sum / static_cast<float>(a.cols);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * 64 * WPR + t) * 8;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rstd * (g[c][i] - h[c][i] * mean);
            if (a.dh) {
                float e[8];
                load8<E, VEC>(static_cast<const T *>(a.dh) + base + col, a.cols - col, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += e[i];
            }
            if (a.dx) store8<E, VEC>(static_cast<T *>(a.dx) + base + col, a.cols - col, d);
        }
    }
    if (a.part) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * 64 * WPR + t) * 8;
            store8<F32, VEC>(a.part + static_cast<size_t>(blockIdx.x) * a.cols + col, a.cols - col, dw[c]);
        }
    }
}

// dw[c] = Σ_p part[p][c], p in order within each of 16 strips, the strips in order.
__global__ __launch_bounds__(1024) void norm_dw_finish_kernel(const float *__restrict__ part, int parts, int cols,
                                                              float *__restrict__ dw) {
    __shared__ float s[16][65];
    const int c = threadIdx.x & 63, strip = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + c;
    const int per = (parts + 15) / 16, lo = strip * per, hi = lo + per < parts ? lo + per : parts;
    float v = 0.0f;
    if (col < cols)
        for (int p = lo; p < hi; ++p) v += part[static_cast<size_t>(p) * cols + col];
    s[strip][c] = v;
    __syncthreads();
    if (strip == 0 && col < cols) {
        for (int i = 1; i < 16; ++i) v += s[i][c];
        dw[col] = v;
    }
}

constexpr int kNormMaxCols = 32768;

// (waves per row, chunks per lane) of a width: one wave up to 1024 columns,
// four up to 8192, sixteen beyond.
template <typename F>
int by_width(int cols, F f) {
    if (cols <= 512) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    if (cols <= 1024) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
    if (cols <= 2048) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    if (cols <= 4096) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
    if (cols <= 8192) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    if (cols <= 16384) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
}

template <typename E, bool MX>
int launch_norm(const NormArgs &a, hipStream_t s) {
    return by_width(a.cols, [&](auto wpr, auto nc) {
        constexpr int WPR = decltype(wpr)::value, NC = decltype(nc)::value;
        constexpr int RPB = WPR >= 4 ? 1 : 4 / WPR;
        const dim3 grid(static_cast<uint32_t>((a.rows + RPB - 1) / RPB)), block(WPR > 4 ? 64 * WPR : 256);
        if (a.cols % 8 == 0) launch_kernel(rms_norm_kernel<E, MX, true, WPR, NC>, grid, block, 0, s, a);
        else launch_kernel(rms_norm_kernel<E, MX, false, WPR, NC>, grid, block, 0, s, a);
        return static_cast<int>(hipGetLastError());
    });
}

// Workgroups of the gradient kernel (about as many as stay resident), each
// with its row of dw partial sums.
int norm_grad_parts(int rows, int cols) {
    const int most = cols <= 1024 ? 2048 : cols <= 8192 ? 512 : 256;
    return rows < most ? rows : most;
}

template <typename E>
int launch_norm_grad(const NormGradArgs &a, hipStream_t s) {
    return by_width(a.cols, [&](auto wpr, auto nc) {
        constexpr int WPR = decltype(wpr)::value, NC = decltype(nc)::value;
        const dim3 grid(static_cast<uint32_t>(norm_grad_parts(a.rows, a.cols))), block(64 * WPR);
        if (a.cols % 8 == 0) launch_kernel(rms_norm_grad_kernel<E, true, WPR, NC>, grid, block, 0, s, a);
        else launch_kernel(rms_norm_grad_kernel<E, false, WPR, NC>, grid, block, 0, s, a);
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
        launch_kernel(norm_dw_finish_kernel, dim3((cols + 63) / 64), dim3(1024), 0, stream,
                      static_cast<const float *>(workspace), rows > 0 ? norm_grad_parts(rows, cols) : 0, cols, dweight);
        if (hipGetLastError() != hipSuccess) return DBF_ERR_HIP;
    }
    return DBF_OK;
}
