// Device helpers of the MXFP4 kernels: loading, scaling and packing blocks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mpg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t mx_u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));

// Words that hold 8 elements.
template <typename T> struct MxPack { static constexpr int WORDS8 = (int)sizeof(T) * 2; };

// 8 elements from x[k0] on as words, zeros from K on. VEC: x is 16-byte
// aligned (k0 is a multiple of 8).
template <typename T, bool VEC>
__device__ __forceinline__ void mx_load8(const T *x, int k0, int K, uint32_t (&u)[MxPack<T>::WORDS8]) {
    if (VEC && k0 + 8 <= K) {
#pragma unroll
        for (int i = 0; i < MxPack<T>::WORDS8 / 4; ++i) {
            const u32x4 v = reinterpret_cast<const u32x4 *>(x + k0)[i];
#pragma unroll
            for (int d = 0; d < 4; ++d)
                u[4 * i + d] = v[d];
        }
    } else if constexpr (sizeof(T) == 2) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k0 + 2 * i < K ? h[k0 + 2 * i] : 0;
            const uint32_t hi = k0 + 2 * i + 1 < K ? h[k0 + 2 * i + 1] : 0;
            u[i] = lo | (hi << 16);
        }
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = k0 + i < K ? w[k0 + i] : 0;
    }
}

__device__ __forceinline__ uint32_t mx_max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(mx_u16x2, a),
                                                                   __builtin_bit_cast(mx_u16x2, b)));
}

// fp32 bits of the magnitude whose 16-bit pattern (sign cleared) is m; fp16's
// NaN and infinity become fp32 ones.
template <typename T>
__device__ __forceinline__ uint32_t mx_bits32(uint32_t m) {
    if constexpr (__is_same(T, _Float16))
        return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m)) & 0x7FFFFFFFu;
    else
        return m << 16;
}

// Largest magnitude of 8 elements as fp32 bits without the sign.
template <typename T>
__device__ __forceinline__ uint32_t mx_amax8(const uint32_t (&u)[MxPack<T>::WORDS8]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = mx_max_u16x2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu);
        m = mx_max_u16x2(m, mx_max_u16x2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
        return mx_bits32<T>(max(m & 0xFFFFu, m >> 16));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, u[i] & 0x7FFFFFFFu);
        return m;
    }
}

// Scale byte of a block from the fp32 bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx_scale_of(uint32_t bits) {
    const uint32_t e = bits >> 23;
    return e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
}

// Codes of two elements into byte SEL of w. s: 2^(scale - 127) as fp32 bits
// scale << 23 (the conversion reads the exponent field only, 0 as 2^-127).
template <typename T, int SEL>
__device__ __forceinline__ uint32_t mx_cvt2(uint32_t w, uint32_t lo, uint32_t hi, float s) {
    if constexpr (__is_same(T, _Float16))
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(mx_f16x2, lo), s, SEL);
    else if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, lo), s, SEL);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(lo), __uint_as_float(hi), s, SEL);
}

// 8 elements -> 8 codes in one word. A block with scale 255 gets codes of
// zero (its values are NaN whatever the codes say).
template <typename T>
__device__ __forceinline__ uint32_t mx_pack8(const uint32_t (&u)[MxPack<T>::WORDS8], uint32_t b) {
    const float s = __uint_as_float(b << 23);
    uint32_t w = 0;
    if constexpr (sizeof(T) == 2) {
        w = mx_cvt2<T, 0>(w, u[0], 0, s);
        w = mx_cvt2<T, 1>(w, u[1], 0, s);
        w = mx_cvt2<T, 2>(w, u[2], 0, s);
        w = mx_cvt2<T, 3>(w, u[3], 0, s);
    } else {
        w = mx_cvt2<T, 0>(w, u[0], u[1], s);
        w = mx_cvt2<T, 1>(w, u[2], u[3], s);
        w = mx_cvt2<T, 2>(w, u[4], u[5], s);
        w = mx_cvt2<T, 3>(w, u[6], u[7], s);
    }
    return b == 255 ? 0u : w;
}

// 32 rows of one word (two columns of a 2-byte type, low half first; one
// column of fp32) -> per column the scale and the 4 words of codes.
template <typename T>
__device__ __forceinline__ void mx_columns(const uint32_t (&v)[32], uint32_t (&b)[4 / sizeof(T)],
                                           uint32_t (&w)[4 / sizeof(T)][4]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 32; ++r)
            m = mx_max_u16x2(m, v[r] & 0x7FFF7FFFu);
        b[0] = mx_scale_of(mx_bits32<T>(m & 0xFFFFu));
        b[1] = mx_scale_of(mx_bits32<T>(m >> 16));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r0 = v[8 * d + 2 * i], r1 = v[8 * d + 2 * i + 1];
                lo[i] = __builtin_amdgcn_perm(r1, r0, 0x05040100u);
                hi[i] = __builtin_amdgcn_perm(r1, r0, 0x07060302u);
            }
            w[0][d] = mx_pack8<T>(lo, b[0]);
            w[1][d] = mx_pack8<T>(hi, b[1]);
        }
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 32; ++r)
            m = max(m, v[r] & 0x7FFFFFFFu);
        b[0] = mx_scale_of(m);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i] = v[8 * d + i];
            w[0][d] = mx_pack8<T>(u, b[0]);
        }
    }
}

// Values of byte SEL of w (two codes) as words: one of a 2-byte type, two of fp32.
// The conversion reads the scale's exponent field only, 0 as 2^-127.
template <typename T, int SEL>
__device__ __forceinline__ void mx_values2(uint32_t w, float s, uint32_t *v) {
    if constexpr (__is_same(T, _Float16)) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, SEL));
    } else if constexpr (__is_same(T, __bf16)) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, SEL));
    } else {
        const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, SEL);
        v[0] = __float_as_uint(f[0]);
        v[1] = __float_as_uint(f[1]);
    }
}

// 8 codes and their scale byte -> 8 values; a scale of 255 makes them NaN.
template <typename T>
__device__ __forceinline__ void mx_unpack8(uint32_t w, uint32_t b, uint32_t (&v)[MxPack<T>::WORDS8]) {
    constexpr int W2 = MxPack<T>::WORDS8 / 4;
    constexpr uint32_t NAN_WORD = __is_same(T, _Float16) ? 0x7E007E00u : __is_same(T, __bf16) ? 0x7FC07FC0u : 0x7FC00000u;
    const float s = __uint_as_float(b << 23);
    mx_values2<T, 0>(w, s, v);
    mx_values2<T, 1>(w, s, v + W2);
    mx_values2<T, 2>(w, s, v + 2 * W2);
    mx_values2<T, 3>(w, s, v + 3 * W2);
#pragma unroll
    for (int d = 0; d < MxPack<T>::WORDS8; ++d)
        v[d] = b == 255 ? NAN_WORD : v[d];
}

}  // namespace mpg
