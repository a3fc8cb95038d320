// Device helpers of the block formats (include/dbf.h, "Block formats"): 32
// consecutive columns of a row share one power-of-two scale byte s (2^(s-127),
// 255 = NaN) and hold e4m3 or e2m1 codes.
#ifndef DBF_MX_DEVICE_H_
#define DBF_MX_DEVICE_H_

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "dbf_internal.h"

namespace dbf {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __builtin_bit_cast(float, b << 16); }

// Element types of the kernels' templates, by the public type codes.
struct F16 {
    using T = uint16_t;
    static constexpr int code = DBF_TYPE_F16;
    __device__ static float get(uint16_t v) { return static_cast<float>(__builtin_bit_cast(_Float16, v)); }
    __device__ static uint16_t put(float v) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)); }
};
struct BF16 {
    using T = uint16_t;
    static constexpr int code = DBF_TYPE_BF16;
    __device__ static float get(uint16_t v) { return bf16_bits_to_float(v); }
    __device__ static uint16_t put(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
};
struct F32 {
    using T = float;
    static constexpr int code = DBF_TYPE_F32;
    __device__ static float get(float v) { return v; }
    __device__ static float put(float v) { return v; }
};

// Eight consecutive elements from p as floats.  VEC: p is aligned to the
// eight elements' size (at most 16 bytes); otherwise element loads, zeros
// from `valid` on (valid may be <= 0 or > 8).
template <typename E, bool VEC>
__device__ __forceinline__ void load8(const typename E::T *p, int valid, float (&v)[8]) {
    if constexpr (VEC) {
        if (valid <= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
            return;
        }
        if constexpr (sizeof(typename E::T) == 2) {
            const u32v4 q = *reinterpret_cast<const u32v4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = E::get(static_cast<uint16_t>(q[i] & 0xffffu));
                v[2 * i + 1] = E::get(static_cast<uint16_t>(q[i] >> 16));
            }
        } else {
            const u32v4 a = reinterpret_cast<const u32v4 *>(p)[0], b = reinterpret_cast<const u32v4 *>(p)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (copies: a bit cast of a vector's element reads element 0)
                const uint32_t lo = a[i], hi = b[i];
                v[i] = __builtin_bit_cast(float, lo);
                v[4 + i] = __builtin_bit_cast(float, hi);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? E::get(p[i]) : 0.0f;
    }
}

// Eight consecutive elements to p, the first `valid` of them (VEC: all or none).
template <typename E, bool VEC>
__device__ __forceinline__ void store8(typename E::T *p, int valid, const float (&v)[8]) {
    if constexpr (VEC) {
        if (valid <= 0) return;
        if constexpr (sizeof(typename E::T) == 2) {
            u32v4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = static_cast<uint32_t>(E::put(v[2 * i])) | static_cast<uint32_t>(E::put(v[2 * i + 1])) << 16;
            *reinterpret_cast<u32v4 *>(p) = q;
        } else {
            u32v4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __builtin_bit_cast(uint32_t, v[i]);
                b[i] = __builtin_bit_cast(uint32_t, v[4 + i]);
            }
            reinterpret_cast<u32v4 *>(p)[0] = a;
            reinterpret_cast<u32v4 *>(p)[1] = b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = E::put(v[i]);
    }
}

// Largest of a value over the four lanes that share a block (lanes 4q..4q+3).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    // quad_perm [1,0,3,2], then [2,3,0,1]
    uint32_t o = __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true);
    v = v > o ? v : o;
    o = __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true);
    return v > o ? v : o;
}

// Largest exponent of a format's values (448 = 1.75 * 2^8, 6 = 1.5 * 2^2).
template <int FMT>
__device__ constexpr int mx_emax() { return FMT == DBF_TYPE_E4M3 ? 8 : 2; }

// Scale byte of a block whose largest magnitude has the float bits `amax`:
// floor(log2 amax) - emax + 127 clamped to [0, 254]; 255 for infinity / NaN.
// The biased exponent of a float is floor(log2) + 127 (0 for subnormals,
// which clamp to 0 either way).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const int e = static_cast<int>(amax >> 23);
    const int s = e - mx_emax<FMT>();
    return e == 255 ? 255u : static_cast<uint32_t>(s > 0 ? s : 0);
}

// 2^(s - 127) as a float: s = 0 is a subnormal, s = 255 a NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
    const uint32_t bits = s == 0 ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23;
    return __builtin_bit_cast(float, bits);
}

// Turn saturation of e4m3 conversions on or off for this wave (the mode bit
// FP16_OVFL; it also keeps overflowing f16 results finite, so it is on only
// around the conversions).
__device__ __forceinline__ void mx_saturate(bool on) {
    // hwreg(MODE, offset 23, size 1)
    if (on) __builtin_amdgcn_s_setreg(1 | (23 << 6), 1);
    else __builtin_amdgcn_s_setreg(1 | (23 << 6), 0);
}

// Codes of eight values of a block with scale byte s: e4m3 in two words,
// e2m1 in one.  The conversion instruction divides by the power of two and
// rounds to nearest even; e2m1 saturates in it, e4m3 under mx_saturate.  A
// block with a non-finite value (s = 255) has zero codes.
template <int FMT>
__device__ __forceinline__ u32v2 mx_codes8(const float (&v)[8], uint32_t s) {
    u32v2 r = {0u, 0u};
    if (s == 255u) return r;
    const float sc = mx_scale_value(s);
    if constexpr (FMT == DBF_TYPE_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s16x2 w = {0, 0};
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[4 * h], v[4 * h + 1], sc, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[4 * h + 2], v[4 * h + 3], sc, true);
            r[h] = __builtin_bit_cast(uint32_t, w);
        }
    } else {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
        r[0] = w;
    }
    return r;
}

// Quantise the eight columns of this lane (lanes 4q..4q+3 hold one block's 32
// columns in order) and store the codes of column `col` (a multiple of 8) of
// a row, and the block's scale byte at `scale`.
template <int FMT>
__device__ __forceinline__ void mx_store8(const float (&v)[8], int col, uint8_t *crow, uint8_t *scale) {
    float top = 0.0f;  // (maximum: a NaN stays)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_elementwise_maximum(top, fabsf(v[i]));
    const uint32_t a = quad_max(__builtin_bit_cast(uint32_t, top) & 0x7fffffffu);
    const uint32_t s = mx_scale_byte<FMT>(a);
    const u32v2 c = mx_codes8<FMT>(v, s);
    if constexpr (FMT == DBF_TYPE_E4M3) *reinterpret_cast<u32v2 *>(crow + col) = c;
    else *reinterpret_cast<uint32_t *>(crow + col / 2) = c[0];
    if ((col & 31) == 0) *scale = static_cast<uint8_t>(s);
}

}  // namespace dbf

#endif  // DBF_MX_DEVICE_H_
