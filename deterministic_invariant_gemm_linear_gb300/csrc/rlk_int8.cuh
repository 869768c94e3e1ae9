// The 8-bit block format: 32 consecutive columns of a row share a power of two 2^(e - 127)
// and hold whole numbers -127 .. 127.  With E the FP32 exponent field of the block's largest
// magnitude, e = max(1, E - 6), so the largest is 64 .. 127.99 steps; E = 255 (a NaN or an
// infinity in the block) gives e = 255 with all q = 0, and 0 * inf reads back as NaN.
//
// A power of two and not max / 127: q 2^(e - 127) is then exact in BF16, so a product that
// reads it is the product of the stored value, with no second rounding; the price is up to
// one bit of the largest magnitudes (half a step is 2^-8 .. 2^-7 of the maximum, against 2^-8).
#pragma once

#include "rlk_device.cuh"

namespace rlk {

constexpr int kInt8Block = 32;

// The larger magnitude; NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}

// The exponent byte from the block's largest magnitude.
__device__ __forceinline__ uint32_t int8_exponent(float most) {
  const int E = (int)(__float_as_uint(most) >> 23 & 255u);
  return E == 255 ? 255u : (uint32_t)max(E - 6, 1);
}
// 2^(127 - e), exact for every e of a finite block (1 .. 248); 0 for e = 255.
__device__ __forceinline__ float int8_inverse(uint32_t e) {
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}
__device__ __forceinline__ float int8_step(uint32_t e) { return __uint_as_float(e << 23); }

// Whether a block with this largest magnitude has values that round to +-128, to be held to +-127
// (|x / step| is below 128, so no others are out of range).  Rare: a call for one branch a block.
__device__ __forceinline__ bool int8_holds(float most, float inverse) {
  return __fmul_rn(most, inverse) >= 127.5f;
}

// Four x / step as bytes, rounded to nearest even, held to -127 .. 127 if `hold`. x / step + 1.5
// 2^23 is rounded to a whole number by the addition (the product is exact), whose low byte it is:
// one fused operation where a conversion would run at a quarter of the rate.
__device__ __forceinline__ uint32_t int8_word(const float* x, float inverse, bool hold) {
  constexpr float kOffset = 12582912.f;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y = __fmaf_rn(x[i], inverse, kOffset);
    if (hold) y = fminf(fmaxf(y, kOffset - 127.f), kOffset + 127.f);
    w[i] = __float_as_uint(y);
  }
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// Four values of a word as FP32: q + 2^23 + 128 built by bytes (q with its sign bit flipped is
// q + 128), then the offset taken off, exactly.
__device__ __forceinline__ void int8_floats(uint32_t word, float step, float* x) {
  word ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 + i));
    x[i] = __fmul_rn(__fsub_rn(v, 8388736.f), step);
  }
}

// Eight values from column c (a multiple of 8) of a row of blocks as FP32; the row begins on 8
// bytes.
__device__ __forceinline__ void load_int8(const int8_t* q, const uint8_t* exponents, int c,
                                          float (&x)[8]) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + c));
  const float step = int8_step(__ldg(exponents + c / kInt8Block));
  int8_floats(w.x, step, x);
  int8_floats(w.y, step, x + 4);
}

}  // namespace rlk
