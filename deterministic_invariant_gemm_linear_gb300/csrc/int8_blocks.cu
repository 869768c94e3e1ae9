// Activations in 8 bits and back (the block format of rlk_int8.cuh).
//
// Both passes are bound by HBM: a BF16 element to 8 bits moves 3.03 bytes (2 read, 1 written,
// an exponent byte per 32), back as much.  A thread takes eight columns, so a block's 32 columns
// lie in four neighbouring lanes: one 16-byte load a thread, the largest magnitude by two
// shuffles, one 8-byte store.
#include "rlk.h"
#include "rlk_int8.cuh"
#include "rlk_internal.h"
#include "rlk_rows.cuh"

namespace rlk {

__device__ unsigned int g_err_int8 = 0;

namespace {

template <bool kFp32>
__global__ void __launch_bounds__(kRowThreads)
    pack_int8_kernel(const void* __restrict__ x, int64_t rows, int cols, int64_t ldx, int vec,
                     int8_t* __restrict__ q, int64_t ldq, uint8_t* __restrict__ exponents,
                     int64_t lde, RowLanes lanes) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t r = (int64_t)blockIdx.x * lanes.rows() + lanes.row();
  const int wide = (cols + kInt8Block - 1) / kInt8Block * kInt8Block;
  // whole warps stay in the loop together: the four lanes of a block exchange maxima
  for (int c0 = 0; c0 < wide; c0 += lanes.step()) {
    const int c = c0 + lanes.col();
    const bool in = r < rows && c < wide;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (in) load8<kFp32>(x, r * ldx, c, cols, vec, v);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    if (!in) continue;
    const uint32_t e = int8_exponent(most);
    const float inverse = int8_inverse(e);
    uint32_t w[2] = {0, 0};
    if (e != 255u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2] |= int8_value(v[i], inverse) << (8 * (i & 3));
    }
    if (RLK_STORE_OK(c + 8 <= ldq, &g_err_int8))
      *reinterpret_cast<uint2*>(q + r * ldq + c) = make_uint2(w[0], w[1]);
    if ((c & (kInt8Block - 1)) == 0 && RLK_STORE_OK(c / kInt8Block < lde, &g_err_int8))
      exponents[r * lde + c / kInt8Block] = (uint8_t)e;
  }
}

template <bool kFp32>
__global__ void __launch_bounds__(kRowThreads)
    unpack_int8_kernel(const int8_t* __restrict__ q, int64_t rows, int cols, int64_t ldq,
                       const uint8_t* __restrict__ exponents, int64_t lde, void* __restrict__ out,
                       int64_t ldo, int vec, RowLanes lanes) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t r = (int64_t)blockIdx.x * lanes.rows() + lanes.row();
  if (r >= rows) return;
  for (int c = lanes.col(); c < cols; c += lanes.step()) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + r * ldq + c));
    const float step = int8_step(__ldg(exponents + r * lde + c / kInt8Block));
    float v[8];
    int8_floats(w.x, step, v);
    int8_floats(w.y, step, v + 4);
    if (RLK_STORE_OK(min(c + 8, cols) <= ldo, &g_err_int8))
      store8<kFp32>(out, r * ldo, c, cols, vec, v);
  }
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
  const RowLanes lanes = row_lanes(cols);
  const dim3 grid((unsigned)ceil_div(rows, lanes.rows()));
  const int vec = rows_vec(x, ldx, dtype_bytes(x_dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((x_dtype == RLK_FP32
           ? launch_overlapped(pack_int8_kernel<true>, grid, kRowThreads, 0, s, x, rows, (int)cols,
                               ldx, vec, q, ldq, exponents, ld_exponents, lanes)
           : launch_overlapped(pack_int8_kernel<false>, grid, kRowThreads, 0, s, x, rows, (int)cols,
                               ldx, vec, q, ldq, exponents, ld_exponents, lanes)) != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return RLK_OK;
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
  const RowLanes lanes = row_lanes(cols);
  const dim3 grid((unsigned)ceil_div(rows, lanes.rows()));
  const int vec = rows_vec(out, ld_out, dtype_bytes(out_dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((out_dtype == RLK_FP32
           ? launch_overlapped(unpack_int8_kernel<true>, grid, kRowThreads, 0, s, q, rows,
                               (int)cols, ldq, exponents, ld_exponents, out, ld_out, vec, lanes)
           : launch_overlapped(unpack_int8_kernel<false>, grid, kRowThreads, 0, s, q, rows,
                               (int)cols, ldq, exponents, ld_exponents, out, ld_out, vec,
                               lanes)) != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return RLK_OK;
}

}  // extern "C"
