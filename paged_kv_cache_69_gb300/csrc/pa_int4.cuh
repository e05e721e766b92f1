// pa_int4.cuh -- the 4-bit cache format: quantising a row and reading codes.
//
// A row is one token's head_dim values of one KV head.  It is held as 4-bit
// codes c in 0..15 and two f16 numbers, step and low:
//     low  = f16(min x)             step = f16((max x - low) / 15)
//     c    = (x - low) / step rounded to nearest even, limited to 0..15
//     x'   = low + step * c
// with x limited to +-65504 first (the largest f16, as fp8 caches limit to
// their largest value), every rounding from the exact value, and c = 0 where
// step is 0 (a row of equal values).  A row that holds a NaN has step = low =
// NaN and reads as NaN throughout.
//
// Layout of one K (or V) block of a pool: codes [num_kv_heads][block_size]
// [head_dim / 2] (dimension 2b in the low nibble of byte b), then (step, low)
// [num_kv_heads][block_size][2] f16.  Heads lie outside the tokens, so the 16
// tokens of a chunk of one head are contiguous (1 KB at head_dim 128), and a
// block is one contiguous span that the block copies and swaps move as bytes.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "pa_device.cuh"

namespace pa {

constexpr int INT4_PARAM_BYTES = 4;           // (step, low) of a row
// The largest value that a f16 output takes.  step may have been rounded up, so
// that a row which reaches 65504 reads as up to 65536 at its top, which f16
// would round to infinity.
constexpr float INT4_F16_TOP = 65504.f;

// Byte offsets of a row's codes and parameters inside its block.
__device__ __forceinline__ uint32_t int4_code_off(int h, int off, int bs, int D) {
    return static_cast<uint32_t>(h * bs + off) * static_cast<uint32_t>(D / 2);
}
__device__ __forceinline__ uint32_t int4_param_off(int h, int off, int bs, int D, int Hkv) {
    return static_cast<uint32_t>(Hkv * bs) * static_cast<uint32_t>(D / 2) +
           static_cast<uint32_t>(h * bs + off) * INT4_PARAM_BYTES;
}

// s = a + b rounded, and the part that the rounding lost (exact).
__device__ __forceinline__ float two_sum(float a, float b, float& lost) {
    const float s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}

// 1 / x to 1 ulp (PTX ISA: rcp.approx.ftz.f32).
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (step, low) of a row with the given extremes.  The quotient a / 15 is
// rounded to odd in f32 before its rounding to f16, so that the two roundings
// give what one from the exact value would: a product with 1 / 15, corrected
// once, is the nearest f32 or next to it, and the residual a - 15 s, exact, says
// on which side the quotient lies.
__device__ __forceinline__ void int4_params(float mn, float mx, __half& step, __half& low) {
    low = __float2half_rn(mn);
    float lost;
    const float a = fmaxf(two_sum(mx, -__half2float(low), lost), 0.f);
    constexpr float R15 = 1.f / 15.f;
    float s = a * R15;
    s = __fmaf_rn(__fmaf_rn(-s, 15.f, a), R15, s);
    const float r = __fadd_rn(__fmaf_rn(-s, 15.f, a), lost);
    uint32_t b = __float_as_uint(s);
    if (s > 0.f && r != 0.f && !(b & 1u)) b += r > 0.f ? 1u : 0xffffffffu;
    step = __float2half_rn(__uint_as_float(b));
}

// The code of x: the nearest of the 16 values, by comparing x with the
// middle between two neighbours.  (c + 1/2) * step has at most 16 bits, so
// the comparison is exact; an estimate of c that is one too low or high next
// to a whole quotient still leads to the right side of it.
__device__ __forceinline__ uint32_t int4_code(float x, float low, float step, float rstep) {
    float lost;
    const float a = two_sum(x, -low, lost);
    const float c = fminf(fmaxf(floorf(a * rstep), 0.f), 15.f);
    const float t = __fadd_rn(__fmaf_rn(-(c + 0.5f), step, a), lost);
    const uint32_t ci = static_cast<uint32_t>(c);
    return min(ci + ((t > 0.f || (t == 0.f && (ci & 1u))) ? 1u : 0u), 15u);
}

// The codes of 8 elements as one word, for r15 = 1 / (15 step).  The quotient
// in plain f32 is off by less than 2^-17 (two roundings of 2^-24 and r15's
// 2^-23, at most 15), so it decides the code unless it lies that near a half; `near`
// then asks for int4_code.  The multiplication saturates to [0, 1], and
// adding 1.5 * 2^23 rounds to the nearest integer and leaves it in the low
// bits, whose constant upper part is taken off the finished word.
__device__ __forceinline__ uint32_t int4_codes8(const float (&x)[8], float low, float r15, float& near) {
    constexpr float MAGIC = 12582912.f;                    // bits 0x4b400000
    uint32_t w = 0;
#pragma unroll
    for (int k = 7; k >= 0; --k) {
        const float q = __saturatef((x[k] - low) * r15);
        const float t = __fmaf_rn(q, 15.f, MAGIC);
        near = fmaxf(near, fabsf(__fmaf_rn(q, 15.f, -__fsub_rn(t, MAGIC))));
        w = w * 16u + __float_as_uint(t);
    }
    return w - 0x4b400000u * 0x11111111u;
}
// Smaller and larger, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// x within f16's largest values, NaN as it is.
__device__ __forceinline__ float limit_f16(float x) { return min_nan(max_nan(x, -INT4_F16_TOP), INT4_F16_TOP); }
constexpr float INT4_NEAR = 0.5f - 1.52587890625e-5f;      // 1/2 - 2^-16

// The value of a code: step * c is exact in f32, the sum is rounded once.
__device__ __forceinline__ float int4_value(uint32_t c, float low, float step) {
    return __fmaf_rn(step, static_cast<float>(c), low);
}

}  // namespace pa
