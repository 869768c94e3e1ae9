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

// The exponent byte from the largest of the block's |x| as FP32 bit patterns (integer order,
// which puts NaN above infinity above every number).
__device__ __forceinline__ uint32_t int8_exponent(uint32_t most_bits) {
  const int E = (int)(most_bits >> 23);
  return E == 255 ? 255u : (uint32_t)max(E - 6, 1);
}
// 2^(127 - e), exact for every e of a finite block (1 .. 248); 0 for e = 255.
__device__ __forceinline__ float int8_inverse(uint32_t e) {
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}
__device__ __forceinline__ float int8_step(uint32_t e) { return __uint_as_float(e << 23); }

// x / step, rounded to nearest even and held to -127 .. 127 (the product is exact).
__device__ __forceinline__ uint32_t int8_value(float x, float inverse) {
  const float q = fminf(fmaxf(__fmul_rn(x, inverse), -127.f), 127.f);
  return (uint32_t)__float2int_rn(q) & 255u;
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

}  // namespace rlk
