// Element-wise passes over the rows of row-major matrices, eight columns a thread: how rows
// and columns are dealt to threads, and loads and stores of eight BF16 or FP32 elements.
#pragma once

#include <cuda_bf16.h>

#include "rlk_device.cuh"
#include "rlk_internal.h"

namespace rlk {

// A block of kRowThreads threads takes `rows()` rows at a time, 1 << shift threads a row (a
// power of two, so that no index is divided), each eight columns and then the ones 8 << shift
// further on.  The eight are runs of kRun consecutive columns (element i at column c + at(i)),
// each run next to the neighbouring lane's, so that a warp's access is one stretch:
//   8   BF16 or 8-bit results, 16-byte vectors
//   4   FP32 results, 16-byte vectors (two of a lane side by side would write half sectors:
//       a 32003 x 2048 table's gradient took 67 us so and takes 40)
//   1   bases, pitches or widths that rule vectors out: single elements
// kRun is a constant of each kernel: a branch around every load would keep the loads of
// several rows from being issued together.
constexpr int kRowThreads = 256;
template <int kRun>
struct RowLanes {
  int shift;
  __host__ __device__ __forceinline__ int rows() const { return kRowThreads >> shift; }
  __host__ __device__ __forceinline__ int step() const { return 8 << shift; }
  __device__ __forceinline__ int row() const { return (int)threadIdx.x >> shift; }
  // columns from one run of a lane to its next
  __device__ __forceinline__ int gap() const { return kRun << (shift < 5 ? shift : 5); }
  __device__ __forceinline__ int col() const {
    const int l = (int)threadIdx.x & ((1 << shift) - 1);
    const int in = l & ((1 << (shift < 5 ? shift : 5)) - 1);
    return 8 * (l - in) + kRun * in;
  }
};
template <int kRun>
inline RowLanes<kRun> row_lanes(int64_t cols, int least_shift = 2) {
  RowLanes<kRun> l{least_shift};
  while (l.shift < 8 && (int64_t(8) << l.shift) < cols) ++l.shift;
  return l;
}
// Column offset of element i.
template <int kRun>
__device__ __forceinline__ int run_at(int i, int gap) {
  return i / kRun * gap + i % kRun;
}

// Whether every row of `esize`-byte elements can be accessed in vectors of n: base, pitch and
// width are whole vectors.
inline bool rows_vec(const void* p, int64_t ld, int64_t esize, int64_t cols, int64_t n) {
  return reinterpret_cast<uintptr_t>(p) % (n * esize < 16 ? n * esize : 16) == 0 &&
         (ld * esize) % (n * esize < 16 ? n * esize : 16) == 0 && cols % n == 0;
}

// The eight elements from column c on (see RowLanes) of a row whose first element is element `at`
// of p; those at or past column n are 0.
template <bool kFp32, int kRun>
__device__ __forceinline__ void load8(const void* p, int64_t at, int c, int gap, int n,
                                      float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / kRun; ++q) {
    const int k = c + q * gap;
    float* y = x + q * kRun;
#pragma unroll
    for (int j = 0; j < kRun; ++j) y[j] = 0.f;
    if (k >= n) continue;
    if constexpr (kRun == 1) {
      if constexpr (kFp32)
        y[0] = __ldg(static_cast<const float*>(p) + at + k);
      else
        y[0] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + at + k) << 16);
    } else if constexpr (kFp32) {
#pragma unroll
      for (int j = 0; j < kRun; j += 4) {
        const float4 a =
            __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + k + j));
        y[j] = a.x; y[j + 1] = a.y; y[j + 2] = a.z; y[j + 3] = a.w;
      }
    } else {
      uint32_t w[kRun / 2];
      const uint16_t* s = static_cast<const uint16_t*>(p) + at + k;
      if constexpr (kRun == 8) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(s));
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(s));
        w[0] = a.x; w[1] = a.y;
      }
#pragma unroll
      for (int j = 0; j < kRun / 2; ++j) {
        y[2 * j] = __uint_as_float(w[j] << 16);
        y[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool kStream, class T>
__device__ __forceinline__ void put(T* p, T v) {
  if constexpr (kStream)
    __stcs(p, v);
  else
    *p = v;
}

// Stores x to the eight columns from c on (those before column n).  kStream: nothing reads them
// soon.
template <bool kFp32, int kRun, bool kStream = false>
__device__ __forceinline__ void store8(void* p, int64_t at, int c, int gap, int n,
                                       const float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / kRun; ++q) {
    const int k = c + q * gap;
    const float* y = x + q * kRun;
    if (k >= n) continue;
    if constexpr (kRun == 1) {
      if constexpr (kFp32)
        static_cast<float*>(p)[at + k] = y[0];
      else
        static_cast<__nv_bfloat16*>(p)[at + k] = __float2bfloat16_rn(y[0]);
    } else if constexpr (kFp32) {
#pragma unroll
      for (int j = 0; j < kRun; j += 4)
        put<kStream>(reinterpret_cast<float4*>(static_cast<float*>(p) + at + k + j),
                     make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]));
    } else {
      uint16_t* d = static_cast<uint16_t*>(p) + at + k;
      if constexpr (kRun == 8)
        put<kStream>(reinterpret_cast<uint4*>(d),
                     make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])));
      else
        put<kStream>(reinterpret_cast<uint2*>(d),
                     make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])));
    }
  }
}

// ---- blocks of 32 x 32 in a warp's registers ----
// An epilogue thread holds 32 columns of its own row.  Where a matrix allows 16-byte vectors it
// writes (or reads) them itself, four neighbouring vectors of one row after another.  Else the
// warp turns its 32 x 32 block by shuffles, so that a lane holds a column, and each row goes out
// as one run of 32 elements: with an odd width every thread would write 32 single elements in a
// row of its own, 32 sectors an instruction in place of two or three (the gated block of 2000 x
// 2048 -> 5461: 140 us, turned 61, as for 5464).

// Element i of lane l <- element (l mod n) of lane l - l mod n + i, n = 32 or 16.
template <int n, class T>
__device__ __forceinline__ void turn_block(T (&x)[n]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = n / 2; s >= 1; s >>= 1) {
    const bool high = lane & s;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if (i & s) continue;
      const T got = __shfl_xor_sync(0xffffffffu, high ? x[i] : x[i | s], s);
      if (high)
        x[i] = got;
      else
        x[i | s] = got;
    }
  }
}

// Columns c .. c + n - 1 (n <= 32) of the warp's rows r0 .. r0 + 31 below M; the whole warp takes
// part, and x, the thread's row, is used up.  vec: whole rows of 32 are 16-byte vectors.  BF16 is
// turned in pairs, columns i and i + 16 in one register: 32 shuffles in place of 80, and a store
// then covers half a row of each half of the block.
template <bool kFp32>
__device__ __forceinline__ void store_block(void* base, int64_t ld, int r0, int M, int c, int n,
                                            bool vec, float (&x)[32]) {
  const int lane = threadIdx.x & 31;
  if (vec && n == 32) {
    if (r0 + lane >= M) return;
    const int64_t at = (int64_t)(r0 + lane) * ld + c;
    if constexpr (kFp32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
      uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                          pack_bf16(x[8 * i + 4], x[8 * i + 5]),
                          pack_bf16(x[8 * i + 6], x[8 * i + 7]));
    }
    return;
  }
  if constexpr (kFp32) {
    turn_block(x);
    float* d = static_cast<float*>(base) + (int64_t)r0 * ld + c + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (r0 + i < M && lane < n) d[i * ld] = x[i];
  } else {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = pack_bf16(x[i], x[i + 16]);
    turn_block(p);
    const int r = r0 + (lane & 16), col = lane & 15;
    uint16_t* d = static_cast<uint16_t*>(base) + (int64_t)r * ld + c + col;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (r + i < M && col < n) d[i * ld] = (uint16_t)p[i];
      if (r + i < M && col + 16 < n) d[i * ld + 16] = (uint16_t)(p[i] >> 16);
    }
  }
}

// Eight consecutive columns a lane (c = those of RowLanes<8>, a whole warp on one row) of rows that
// rule vectors out: the warp reads or writes whole runs of single elements, and the lanes'
// eights change hands through 1 KB of shared memory a warp.  All lanes take part; `in` says
// whether the warp's row exists.
struct RowStage {
  float* buf;                         // this warp's 256 floats
  __device__ __forceinline__ explicit RowStage(float (*all)[256]) : buf(all[threadIdx.x >> 5]) {}
  template <bool kFp32>
  __device__ __forceinline__ void load(const void* p, int64_t at, int c, int n, bool in,
                                       float (&x)[8]) const {
    const int lane = threadIdx.x & 31, c0 = c - 8 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = c0 + 32 * i + lane;
      float v = 0.f;
      if (in && k < n) {
        if constexpr (kFp32)
          v = __ldg(static_cast<const float*>(p) + at + k);
        else
          v = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + at + k) << 16);
      }
      x[i] = v;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[32 * i + lane] = x[i];
    __syncwarp();
    const float4 a = reinterpret_cast<const float4*>(buf)[2 * lane];
    const float4 b = reinterpret_cast<const float4*>(buf)[2 * lane + 1];
    __syncwarp();
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  template <bool kFp32>
  __device__ __forceinline__ void store(void* p, int64_t at, int c, int n, bool in,
                                        const float (&x)[8]) const {
    const int lane = threadIdx.x & 31, c0 = c - 8 * lane;
    reinterpret_cast<float4*>(buf)[2 * lane] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(buf)[2 * lane + 1] = make_float4(x[4], x[5], x[6], x[7]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = c0 + 32 * i + lane;
      if (in && k < n) {
        if constexpr (kFp32)
          static_cast<float*>(p)[at + k] = buf[32 * i + lane];
        else
          static_cast<__nv_bfloat16*>(p)[at + k] = __float2bfloat16_rn(buf[32 * i + lane]);
      }
    }
    __syncwarp();
  }
};

// f(d1, d2, run) with ::value: whether each dtype is FP32, and the run length, as constants.
template <auto kValue>
struct Const {
  static constexpr auto value = kValue;
};
template <class F>
inline cudaError_t by_dtypes(int d1, int d2, F f) {
  if (d1 == RLK_FP32)
    return d2 == RLK_FP32 ? f(Const<true>(), Const<true>()) : f(Const<true>(), Const<false>());
  return d2 == RLK_FP32 ? f(Const<false>(), Const<true>()) : f(Const<false>(), Const<false>());
}

inline bool known_dtype(int d) { return d == RLK_BF16 || d == RLK_FP32; }
inline int dtype_bytes(int d) { return d == RLK_FP32 ? 4 : 2; }
inline bool is_aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
constexpr int64_t kPitchLimit = int64_t(1) << 36;   // leading dimensions, exclusive

}  // namespace rlk
