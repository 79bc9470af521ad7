// The rows of a 4-bit KV cache, shared by the append, the attention and the unpacking.
//
// A row holds one token of one kv head, K and V together, so that a tile of a cache (or
// a block of a pool) is one contiguous copy.  Each half (K, then V) is head_dim 4-bit
// codes followed by one (m, s) pair of bf16 per group of 32 dims; dim i of the half
// stands for code_i * s + m with
//     m = the group's smallest value, rounded down to bf16
//     s = (the group's largest value - m) / 15, rounded up to bf16
//     code = rint((x - m) / s), half to even, in [0, 15]   (0 where s = 0)
// so that |x - (code s + m)| <= s / 2 up to fp32 rounding.  m is exact when x is bf16.
// A non-finite x makes m or s, and with them the whole group's values, non-finite.
//
// Codes are 32-bit words w[t][grp] (t = 0..3, grp = 0..head_dim/32-1): nibble n of the
// word is dim 32 grp + 8 t + n.  A lane that owns word column t of a row so reads the
// codes of every group with one load, and the even / odd nibbles of a word's low and
// (shifted) high halves are, as they stand, fp16 subnormals (code * 2^-24, code * 2^-20).
#pragma once

#include "common.cuh"

namespace sk {

struct Kv4 {};  // tag: a cache of 4-bit rows

constexpr int kv4_row_bytes(int D) { return D + D / 4; }    // K and V
constexpr int kv4_half_bytes(int D) { return D / 2 + D / 8; }
constexpr int kv4_word_offset(int D, int t, int grp) { return t * (D / 8) + grp * 4; }
constexpr int kv4_param_offset(int D, int grp) { return D / 2 + grp * 4; }

// Largest bf16 value <= x, smallest bf16 value >= x (x >= 0), as floats.
__device__ __forceinline__ float bf16_floor(float x) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float((int32_t(b) >= 0 ? b : b + 0xFFFFu) & 0xFFFF0000u);
}

__device__ __forceinline__ float bf16_ceil_nonneg(float x) {
    return x != x ? x : __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u);
}

// Extremes that keep a NaN (fminf / fmaxf drop it, and a group would hide it).
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// x / d for a divisor whose reciprocal is held in two parts, inv + lo = 1/d to 2^-46: one
// rounding of a product that is off by 2^-46, so the quotient is the correctly rounded one
// unless x / d is that close to the middle of two floats, and exact where x / d is a float
// (the ties of rint, and quotients that are bf16 values, among them).
__device__ __forceinline__ float div_by(float x, float inv, float lo) { return fmaf(x, inv, x * lo); }

// (m, s) of a group with extremes lo and hi.
__device__ __forceinline__ void kv4_group_params(float lo, float hi, float* m, float* s) {
    constexpr float inv15 = 1.0f / 15.0f;                        // nearest float
    constexpr float lo15 = float(1.0 / 15.0 - double(inv15));
    *m = bf16_floor(lo);
    *s = bf16_ceil_nonneg(div_by(hi - *m, inv15, lo15));
}

// The pair as stored: m in the low half of the word, s in the high half.
__device__ __forceinline__ uint32_t kv4_param_word(float m, float s) {
    return (__float_as_uint(m) >> 16) | (__float_as_uint(s) & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t kv4_code(float x, float m, float s) {
    const float r = rintf(__fdiv_rn(x - m, s));       // NaN where s is 0 or not finite
    return uint32_t(fminf(fmaxf(r, 0.0f), 15.0f));    // NaN -> 0
}

// Codes of N (4 or 8) values of a group as nibbles 0 .. N - 1.  Where s is neither tiny nor
// huge the quotients are products with 1/s (div_by), in [0, 15] because s was rounded up.
// Adding 1.5 * 2^23 rounds them (half to even) and leaves the code in the low bits under a
// constant, and the constants of all nibbles are taken off the sum at once.
template <int N>
__device__ __forceinline__ uint32_t kv4_codes(const float* x, float m, float s) {
    uint32_t w = 0;
    if (s >= 7.9e-31f && s <= 1.2e27f) {  // 2^-100, 2^90: no part of 1/s underflows
        float inv;  // to 1 ulp; with lo = (1 - s inv) inv the two parts are 1/s to 2^-46
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        const float lo = fmaf(-s, inv, 1.0f) * inv;
        const float2 m2 = make_float2(-m, -m), inv2 = make_float2(inv, inv), lo2 = make_float2(lo, lo);
        const float2 magic = make_float2(12582912.0f, 12582912.0f);
        constexpr uint32_t kMagicSum = 0x4B400000u * (N == 8 ? 0x11111111u : 0x1111u);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 t = __fadd2_rn(make_float2(x[i], x[i + 1]), m2);
            const float2 y = __fadd2_rn(__ffma2_rn(t, inv2, __fmul2_rn(t, lo2)), magic);
            w += (__float_as_uint(y.x) << (4 * i)) + (__float_as_uint(y.y) << (4 * i + 4));
        }
        return w - kMagicSum;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) w |= kv4_code(x[i], m, s) << (4 * i);
    return w;
}

// The 8 values of a word.  A nibble masked in place under the exponent of 2^23 is 2^23 +
// code * 16^i, exactly, for i < 4; the power of 16 goes into the scale.
__device__ __forceinline__ void kv4_decode_word(uint32_t w, uint32_t param, float* f) {
    const float m = __uint_as_float(param << 16), s = __uint_as_float(param & 0xFFFF0000u);
    const float2 m2 = make_float2(m, m), bias = make_float2(-8388608.0f, -8388608.0f);
    const float2 s01 = make_float2(s, s * 0.0625f), s23 = make_float2(s * 0.00390625f, s * 0.000244140625f);
#pragma unroll
    for (int h = 0; h < 2; ++h, w >>= 16) {
        const float2 c01 = __fadd2_rn(make_float2(__uint_as_float((w & 0x000Fu) | 0x4B000000u),
                                                  __uint_as_float((w & 0x00F0u) | 0x4B000000u)), bias);
        const float2 c23 = __fadd2_rn(make_float2(__uint_as_float((w & 0x0F00u) | 0x4B000000u),
                                                  __uint_as_float((w & 0xF000u) | 0x4B000000u)), bias);
        const float2 a = __ffma2_rn(c01, s01, m2), b = __ffma2_rn(c23, s23, m2);
        f[4 * h] = a.x;
        f[4 * h + 1] = a.y;
        f[4 * h + 2] = b.x;
        f[4 * h + 3] = b.y;
    }
}

}  // namespace sk
