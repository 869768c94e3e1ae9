// Activations in 8 bits and back (the block format of rlk_int8.cuh).
//
// A BF16 element to 8 bits moves 3.03 bytes (2 read, 1 written, an exponent byte per 32), back as
// much.  16384 x 4096: packing 38 - 44 us (5.0 TB/s; two thirds of it instructions), unpacking 32 -
// 35 (6.1 TB/s).  A thread takes eight columns, so a block's 32 columns lie in four neighbouring
// lanes: one 16-byte load a thread, the largest magnitude by two shuffles, one 8-byte store.
#include "rlk.h"
#include "rlk_int8.cuh"
#include "rlk_internal.h"
#include "rlk_rows.cuh"

namespace rlk {

__device__ unsigned int g_err_int8 = 0;

namespace {

// kRowsAThread rows a thread, their loads issued together (16384 x 4096 BF16, us with 1, 2, 3 and
// 4: packing 41.6, 37.1, 35.7, 42.3, unpacking 41.1, 36.1, 44.6, 50.1).  Rows that rule vectors out
// (kVec false) pass through shared memory (RowStage).  Packing is bound by instructions as much as
// by HBM.
constexpr int kRowsAThread = 2;

template <bool kFp32, bool kVec>
__global__ void __launch_bounds__(kRowThreads)
    pack_int8_kernel(const void* __restrict__ x, int64_t rows, int cols, int64_t ldx,
                     int8_t* __restrict__ q, int64_t ldq, uint8_t* __restrict__ exponents,
                     int64_t lde, RowLanes<8> lanes) {
  __shared__ __align__(16) float staged[kVec ? 1 : kRowThreads / 32][256];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t r0 = (int64_t)blockIdx.x * (kRowsAThread * lanes.rows()) + lanes.row();
  const int wide = (cols + kInt8Block - 1) / kInt8Block * kInt8Block;
  // whole warps stay in the loop together: a block's four lanes exchange their largest magnitude
  for (int c0 = (int)blockIdx.y * lanes.step(); c0 < wide; c0 += (int)gridDim.y * lanes.step()) {
    const int c = c0 + lanes.col();
    float v[kRowsAThread][8];
#pragma unroll
    for (int k = 0; k < kRowsAThread; ++k) {
      const int64_t r = r0 + k * lanes.rows();
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
      if constexpr (kVec) {
        if (r < rows) load8<kFp32, 8>(x, r * ldx, c, 0, cols, v[k]);
      } else {
        RowStage(staged).load<kFp32>(x, r * ldx, c, cols, r < rows, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsAThread; ++k) {
      const int64_t r = r0 + k * lanes.rows();
      float most = fabsf(v[k][0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) most = max_magnitude(most, v[k][i]);
      most = max_magnitude(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max_magnitude(most, __shfl_xor_sync(0xffffffffu, most, 2));
      if (r >= rows || c >= wide ||
          !RLK_STORE_OK(c + 8 <= ldq && c / kInt8Block < lde, &g_err_int8))
        continue;
      const uint32_t e = int8_exponent(most);
      const float inverse = int8_inverse(e);
      uint2 w;
      if (int8_holds(most, inverse))
        w = make_uint2(int8_word(v[k], inverse, true), int8_word(v[k] + 4, inverse, true));
      else
        w = make_uint2(int8_word(v[k], inverse, false), int8_word(v[k] + 4, inverse, false));
      if (e == 255u) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(q + r * ldq + c) = w;
      if ((c & (kInt8Block - 1)) == 0) exponents[r * lde + c / kInt8Block] = (uint8_t)e;
    }
  }
}

// kRun 8: BF16 in vectors, 4: FP32 in vectors, 1: by way of shared memory.
template <bool kFp32, int kRun>
__global__ void __launch_bounds__(kRowThreads)
    unpack_int8_kernel(const int8_t* __restrict__ q, int64_t rows, int cols, int64_t ldq,
                       const uint8_t* __restrict__ exponents, int64_t lde, void* __restrict__ out,
                       int64_t ldo, RowLanes<kRun == 4 ? 4 : 8> lanes) {
  __shared__ __align__(16) float staged[kRun == 1 ? kRowThreads / 32 : 1][256];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t r0 = (int64_t)blockIdx.x * (kRowsAThread * lanes.rows()) + lanes.row();
  const int gap = lanes.gap();
  for (int c0 = (int)blockIdx.y * lanes.step(); c0 < cols; c0 += (int)gridDim.y * lanes.step()) {
    const int c = c0 + lanes.col();
    float v[kRowsAThread][8];
#pragma unroll
    for (int k = 0; k < kRowsAThread; ++k) {
      const int64_t r = r0 + k * lanes.rows();
      if (r >= rows) continue;
      const int8_t* values = q + r * ldq;
      const uint8_t* e = exponents + r * lde;
      if constexpr (kRun == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = c + h * gap;
          if (at < cols)
            int8_floats(__ldg(reinterpret_cast<const uint32_t*>(values + at)),
                        int8_step(__ldg(e + at / kInt8Block)), v[k] + 4 * h);
        }
      } else if (c < cols) {
        load_int8(values, e, c, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsAThread; ++k) {
      const int64_t r = r0 + k * lanes.rows();
      const bool in = r < rows && RLK_STORE_OK(cols <= ldo, &g_err_int8);
      if constexpr (kRun == 1)
        RowStage(staged).store<kFp32>(out, r * ldo, c, cols, in, v[k]);
      else if (in)
        store8<kFp32, kRun>(out, r * ldo, c, gap, cols, v[k]);
    }
  }
}

// Rows to blocks, and their column steps too (the y dimension's limit aside).
template <int kRun>
dim3 int8_grid(int64_t rows, int64_t cols, const RowLanes<kRun>& lanes) {
  const int64_t steps = ceil_div(cols, lanes.step());
  return dim3((unsigned)ceil_div(rows, kRowsAThread * lanes.rows()),
              (unsigned)(steps < 65535 ? steps : 65535));
}

// Column extents stay below 2^30: a thread's column index plus a step must fit an int.
constexpr int64_t kMaxCols = int64_t(1) << 30;

rlk_status check_int8(int dtype, int64_t rows, int64_t cols, int64_t ld, int64_t ldq, int64_t lde) {
  if (!known_dtype(dtype)) return RLK_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxExtent || cols < 1 || cols >= kMaxCols || ld < cols ||
      ld >= kPitchLimit || ldq < ceil_div(cols, kInt8Block) * kInt8Block || ldq % 16 != 0 ||
      ldq >= kPitchLimit || lde < ceil_div(cols, kInt8Block) || lde >= kPitchLimit)
    return RLK_ERR_SHAPE;
  return RLK_OK;
}

rlk_status cuda_failed() {
  cudaGetLastError();
  return RLK_ERR_CUDA;
}

}  // namespace

uint32_t take_error_int8() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_int8, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaMemcpyToSymbol(g_err_int8, &zero, sizeof zero);
  cudaGetLastError();
  return v;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_pack_int8(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                         int8_t* q, int64_t ldq, uint8_t* exponents, int64_t ld_exponents,
                         void* stream) {
  RLK_CALL_RANGE();
  rlk_status st = check_int8(x_dtype, rows, cols, ldx, ldq, ld_exponents);
  if (st != RLK_OK) return st;
  if (rows == 0) return RLK_OK;
  if (!x || !q || !exponents) return RLK_ERR_NULL;
  if (!is_aligned(x, dtype_bytes(x_dtype)) || !is_aligned(q, 16)) return RLK_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  const bool vec = rows_vec(x, ldx, dtype_bytes(x_dtype), cols, 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto launch = [&](auto x32, auto v) {
    constexpr bool kVec = decltype(v)::value;
    const RowLanes<8> lanes = row_lanes<8>(cols, kVec ? 2 : 5);
    return launch_overlapped(pack_int8_kernel<decltype(x32)::value, kVec>,
                             int8_grid(rows, cols, lanes), kRowThreads, 0, s, x, rows, (int)cols,
                             ldx, q, ldq, exponents, ld_exponents, lanes);
  };
  const auto by_vec = [&](auto x32) {
    return vec ? launch(x32, Const<true>()) : launch(x32, Const<false>());
  };
  return (x_dtype == RLK_FP32 ? by_vec(Const<true>()) : by_vec(Const<false>())) == cudaSuccess
             ? RLK_OK
             : cuda_failed();
}

rlk_status rlk_unpack_int8(const int8_t* q, int64_t rows, int64_t cols, int64_t ldq,
                           const uint8_t* exponents, int64_t ld_exponents, void* out,
                           int out_dtype, int64_t ld_out, void* stream) {
  RLK_CALL_RANGE();
  rlk_status st = check_int8(out_dtype, rows, cols, ld_out, ldq, ld_exponents);
  if (st != RLK_OK) return st;
  if (rows == 0) return RLK_OK;
  if (!q || !exponents || !out) return RLK_ERR_NULL;
  if (!is_aligned(out, dtype_bytes(out_dtype)) || !is_aligned(q, 16)) return RLK_ERR_ALIGN;
  DeviceInfo dev;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  const bool fp32 = out_dtype == RLK_FP32;
  const bool vec = rows_vec(out, ld_out, dtype_bytes(out_dtype), cols, fp32 ? 4 : 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto launch = [&](auto o32, auto run) {
    constexpr int kRun = decltype(run)::value;
    const auto lanes = row_lanes<kRun == 4 ? 4 : 8>(cols, kRun == 1 ? 5 : 2);
    return launch_overlapped(unpack_int8_kernel<decltype(o32)::value, kRun>,
                             int8_grid(rows, cols, lanes), kRowThreads, 0, s, q, rows, (int)cols,
                             ldq, exponents, ld_exponents, out, ld_out, lanes);
  };
  const cudaError_t e =
      fp32 ? vec ? launch(Const<true>(), Const<4>()) : launch(Const<true>(), Const<1>())
      : vec ? launch(Const<false>(), Const<8>())
            : launch(Const<false>(), Const<1>());
  return e == cudaSuccess ? RLK_OK : cuda_failed();
}

}  // extern "C"
