// Element-wise passes over the rows of row-major matrices, eight columns a thread: how rows
// and columns are dealt to threads, and loads and stores of eight BF16 or FP32 elements.
#pragma once

#include <cuda_bf16.h>

#include "rlk_device.cuh"
#include "rlk_internal.h"

namespace rlk {

// A block of kRowThreads threads takes `rows()` rows at a time, 1 << shift threads a row (a
// power of two, so that no index is divided), each eight columns and then the ones 8 << shift
// further on.
constexpr int kRowThreads = 256;
struct RowLanes {
  int shift;
  __host__ __device__ __forceinline__ int rows() const { return kRowThreads >> shift; }
  __device__ __forceinline__ int row() const { return (int)threadIdx.x >> shift; }
  __device__ __forceinline__ int col() const { return ((int)threadIdx.x & ((1 << shift) - 1)) * 8; }
  __host__ __device__ __forceinline__ int step() const { return 8 << shift; }
};
inline RowLanes row_lanes(int64_t cols) {
  RowLanes l{2};
  while (l.shift < 8 && (int64_t(8) << l.shift) < cols) ++l.shift;
  return l;
}

// Whether rows of `esize`-byte elements can be read or written eight at a time with 16-byte
// vectors: base and pitch are multiples of 16 bytes.
inline bool rows_vec(const void* p, int64_t ld, int64_t esize) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esize) % 16 == 0;
}

// Elements c .. c + 7 of a row whose first element is element `at` of p; those at or past
// column n are 0.
template <bool kFp32>
__device__ __forceinline__ void load8(const void* p, int64_t at, int c, int n, bool vec,
                                      float (&x)[8]) {
  if (vec && c + 8 <= n) {
    if constexpr (kFp32) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + c);
      const float4 a = __ldg(s), b = __ldg(s + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint4 a =
          __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at + c));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = 0.f;
    if (c + i < n) {
      if constexpr (kFp32)
        x[i] = __ldg(static_cast<const float*>(p) + at + c + i);
      else
        x[i] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + at + c + i) << 16);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Stores x to elements c .. c + 7 of the row (those before column n).
template <bool kFp32>
__device__ __forceinline__ void store8(void* p, int64_t at, int c, int n, bool vec,
                                       const float (&x)[8]) {
  if (vec && c + 8 <= n) {
    if constexpr (kFp32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at + c);
      d[0] = make_float4(x[0], x[1], x[2], x[3]);
      d[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at + c) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) {
      if constexpr (kFp32)
        static_cast<float*>(p)[at + c + i] = x[i];
      else
        static_cast<__nv_bfloat16*>(p)[at + c + i] = __float2bfloat16_rn(x[i]);
    }
}

// f(a, b) with a::value, b::value: whether each dtype is FP32, as constants.
template <bool kValue>
struct BoolC {
  static constexpr bool value = kValue;
};
template <class F>
inline cudaError_t by_dtypes(int d1, int d2, F f) {
  if (d1 == RLK_FP32) return d2 == RLK_FP32 ? f(BoolC<true>(), BoolC<true>()) : f(BoolC<true>(), BoolC<false>());
  return d2 == RLK_FP32 ? f(BoolC<false>(), BoolC<true>()) : f(BoolC<false>(), BoolC<false>());
}

inline bool known_dtype(int d) { return d == RLK_BF16 || d == RLK_FP32; }
inline int dtype_bytes(int d) { return d == RLK_FP32 ? 4 : 2; }
inline bool is_aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
constexpr int64_t kPitchLimit = int64_t(1) << 36;   // leading dimensions, exclusive

}  // namespace rlk
