// The gated linear block on sm_103a: both projections, the gate's activation and the product in
// one kernel, and its backward.
//
//   g = X . Wg^T,  u = X . Wu^T,  h = act(g) u        act(g) = g s,  s = sigmoid(a(g))
//   SiLU: a(g) = g;  GELU in its tanh form: a(g) = 2 sqrt(2/pi) (g + 0.044715 g^3)
//   act'(g) = s + g s (1 - s) a'(g)
//   G = dL/d[g, u] = [d u act'(g), d act(g)],  dX = G . W,  dW = G^T . X        W = [Wg; Wu]
//
// The forward is 4 M K F operations on the tensor cores.  A tile of 256 rows holds 128 columns of g
// and the same 128 of u side by side in one accumulator (MMA N = 256): the right operand's tile is
// 128 rows of Wg followed by 128 of Wu, read by one 3-D tensor map {K, F, 2}.  So the loops are
// the library's (rlk_pipeline.cuh, rlk_solo.cuh), each accumulator is the sum that det_linear
// forms, and the epilogue thread that owns a row finds g and u of a column 128 accumulator columns
// apart: the [M, 2 F] projections need not exist.
// The backward forms G (the same loop again, or one pass over kept g and u), rounds it to BF16,
// the type in which the two products read it, and runs them as det_linear's backward.
#include <math.h>

#include <mutex>

#include <cuda_bf16.h>

#include "rlk.h"
#include "rlk_int8.cuh"
#include "rlk_internal.h"
#include "rlk_pipeline.cuh"
#include "rlk_rows.cuh"
#include "rlk_solo.cuh"

namespace rlk {

__device__ unsigned int g_err_gated_linear = 0;

namespace {

constexpr int kGateCols = kBN / 2;     // columns of g (and of u) in a 256-wide accumulator
// Eight epilogue warps, two to a quarter of the accumulator rows, each half of a tile's columns: one
// warp a scheduler issues an instruction in four cycles.  Four warps / eight, us: forward of 2000 x
// 512 -> 4000 19.4 / 18.7, with 8 bits kept 31.6 / 26.6, its backward with G from projections formed
// again 87.6 / 77.0; 4096 x 1024 -> 4096 37.6 / 38.0, 56.4 / 50.3, 164 / 143; 2000 x 2048 -> 5464, whose
// MMAs hide either, 51.7 / 52.4, 58.6 / 59.9, 180 / 175.
constexpr int kEpilogueWarps = 8;
constexpr int kGatedThreads = 64 + 32 * kEpilogueWarps;     // and the producer's and the MMAs' warp
constexpr int kSlotBytes = 4096;       // a block of 32 x 32 FP32 on its way out (see StoreSlots)
constexpr int kStoreBytes = kEpilogueWarps * kSlotBytes;

// ---------------------------------------------------------------- the activation
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kTanhSlope = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

// s = sigmoid(a(g)) and s (1 - s), from e = exp(-|a|) so that neither overflows.  In FP32: the
// argument's roundings make e off by up to 3 |a| 2^-23, the two approximations and the products
// add 2^-21 (2^-14 in all for a of -87, far below a BF16 result's half step); below the normal
// numbers (a under -87.3) e and with it s are 0.
template <int kAct>
__device__ __forceinline__ void gate(float g, float& s, float& both) {
  float a = g;
  if constexpr (kAct == RLK_ACT_GELU_TANH)
    a = kTanhSlope * __fmaf_rn(kTanhCube * g * g, g, g);
  const float e = ex2_approx(-fabsf(a) * kLog2e);
  const float r = rcp_approx(1.f + e);
  s = a < 0.f ? e * r : r;
  both = e * r * r;
}

template <int kAct>
__device__ __forceinline__ float gate_value(float g) {
  float s, both;
  gate<kAct>(g, s, both);
  return g * s;
}

// act(g) and act'(g).
template <int kAct>
__device__ __forceinline__ void gate_slope(float g, float& value, float& slope) {
  float s, both;
  gate<kAct>(g, s, both);
  value = g * s;
  float da = 1.f;
  if constexpr (kAct == RLK_ACT_GELU_TANH)
    da = kTanhSlope * __fmaf_rn(3.f * kTanhCube * g, g, 1.f);
  slope = both == 0.f ? s : __fmaf_rn(g * both, da, s);   // a flat end, however large a'(g)
}

// ---------------------------------------------------------------- operands and schedule
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar, int32_t c0, int32_t c1,
                                                 int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The right operand of the 2-SM loop.  The loop asks for rows [row0, row0 + 128) of tiles of 256:
// tile t is columns [128 t, 128 t + 128) of g, whose weight rows rank 0 stages, and the same of
// u, whose rows rank 1 stages.  K-major, laid out as OperandTile<false, 128>.
template <int kStageK>
struct GateUpHalf {
  using Layout = OperandTile<false, kGateCols, kStageK>;
  static constexpr int kK = kStageK;
  static constexpr uint32_t kBytes = Layout::kBytes;
  template <bool kPair>
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t row0, int32_t k0) {
    const int32_t f0 = row0 / (2 * kGateCols) * kGateCols, plane = row0 / kGateCols & 1;
#pragma unroll
    for (int i = 0; i < kStageK / 64; ++i)
      tma_load_3d_pair(dst + i * (kGateCols * 128), map, bar, k0 + 64 * i, f0, plane);
  }
  static __device__ __forceinline__ uint64_t desc(uint32_t base, int kstep) {
    return Layout::desc(base, kstep);
  }
};

// The right operand of the one-CTA loop: kCols rows of Wg, then the same of Wu, in one copy.
template <int kCols>
struct GateUpBoth {
  using Layout = OperandTile<false, 2 * kCols>;
  static constexpr uint32_t kBytes = Layout::kBytes;
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t row0, int32_t k0) {
    tma_load_3d(dst, map, bar, k0, row0 / 2, 0);
  }
  static __device__ __forceinline__ uint64_t desc(uint32_t base, int kstep) {
    return Layout::desc(base, kstep);
  }
};

// The 2-SM loop's ring, with room for the epilogue's store slots after it (3 stages of 128
// reduction elements, or 6 of 64).
template <int kK>
using GatedRing = PairRingT<kHalfRows, kK, kStoreBytes>;

struct GatedSched {
  Banded order;     // rows = blocks of 256 rows (one CTA pair) or the only one of 128, cols = tiles
  int* counter;     // zeroed unit counter in the workspace, or null (round-robin)
  int nkb, nkb64;   // reduction stages over K, and its 64-wide blocks
  int tile_rows;    // right-operand rows per tile: 256, or 2 w in the one-CTA loop
  __device__ __forceinline__ int num_units() const { return order.count(); }
  __device__ __forceinline__ int unit_tiles(int) const { return 1; }
  __device__ __forceinline__ void tile_coords(int u, int, int& a0, int& b0) const {
    int rb, ct;
    order.unit(u, rb, ct);
    a0 = rb * kPairRows;
    b0 = ct * tile_rows;
  }
};

// A block of 32 x 32 (see store_block) read: x is the thread's row, 0 past column n and past row M.
// The turned loads take the block's nearest element where there is none, so that none hangs on a
// branch (with branches the 32 loads came one after another: G of 2000 x 5461 158 us, without 80).
template <bool kFp32>
__device__ __forceinline__ void load_block(const void* base, int64_t ld, int r0, int M, int c,
                                           int n, bool vec, float (&x)[32]) {
  const int lane = threadIdx.x & 31;
  const bool in = r0 + lane < M;
  if (vec && n == 32) {
    const int64_t at = (int64_t)(in ? r0 + lane : M - 1) * ld + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[8];
      load8<kFp32, 8>(base, at, 8 * i, 0, 32, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[8 * i + j] = y[j];
    }
  } else if constexpr (kFp32) {
    const float* s = static_cast<const float*>(base) + c + min(lane, n - 1);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __ldg(s + (int64_t)min(r0 + i, M - 1) * ld);
    turn_block(x);
  } else {
    uint32_t p[16];
    const int r = r0 + (lane & 16), col = lane & 15;
    const uint16_t* s = static_cast<const uint16_t*>(base) + c;
    const int lo = min(col, n - 1), hi = min(col + 16, n - 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint16_t* row = s + (int64_t)min(r + i, M - 1) * ld;
      p[i] = (uint32_t)__ldg(row + lo) | (uint32_t)__ldg(row + hi) << 16;
    }
    turn_block(p);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = __uint_as_float(p[i] << 16);
      x[i + 16] = __uint_as_float(p[i] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!in || i >= n) x[i] = 0.f;
}

inline bool block_vec(const void* base, int64_t ld, int64_t esize) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (ld * esize) % 16 == 0;
}

// Blocks of 32 rows and 32 columns on their way out by TMA.  A warp has 4 KB after the ring's stages:
// room for one block of FP32, or for two of BF16 or bytes.  Each thread writes its row (16-byte
// pieces swizzled as the tensor map says, so that no two lanes of a phase share a bank), lane 0
// starts the copy and the warp goes on; the room is taken again once the copy has been read.  The
// copies write whole rows of 32, 64 or 128 bytes and end at the matrix's last row by themselves.
// (Not at its last column: a box that the width cuts is written in units of 16 bytes, so a run of
// fewer than 32 columns goes out from the threads.)  Against stores from the threads, 16 bytes in
// each of 32 rows an instruction (four epilogue warps, FP32 projections kept): 4096 x 64 -> 16384
// 157 us for 267, 4096 x 4096 -> 16384 595 for 622.
struct StoreSlots {
  uint32_t base;             // this warp's 4 KB, or 0 (stores from the threads)
  uint32_t at;               // where the next block is put
  bool whole = false;        // the last block had all of it
  __device__ __forceinline__ explicit StoreSlots(uint32_t b) : base(b), at(b) {}
  // Room for a block of FP32 (kWhole), or of BF16 or bytes.
  template <bool kWhole>
  __device__ __forceinline__ uint32_t take() {
    if ((threadIdx.x & 31) == 0) {
      if (kWhole || whole)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      else
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    }
    __syncwarp();
    at = kWhole || at != base ? base : base + kSlotBytes / 2;
    whole = kWhole;
    return at;
  }
  // Sends it to columns c .. c + 31 of rows r .. r + 31.
  __device__ __forceinline__ void send(const CUtensorMap* map, int c, int r) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      asm volatile(
          "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
              reinterpret_cast<uint64_t>(map)),
          "r"(at), "r"(c), "r"(r)
          : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  // Every copy has been written (before the CTA gives up its shared memory).
  __device__ __forceinline__ void finish() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
};

__device__ __forceinline__ void put16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// Row `lane` of a slot: 32 FP32 patterns, 32 numbers as BF16, or 32 bytes.
__device__ __forceinline__ void put_fp32(uint32_t slot, const uint32_t (&x)[32]) {
  const uint32_t r = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    put16(slot + 128 * r + 16 * (i ^ (r & 7)), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void put_bf16(uint32_t slot, const float (&x)[32]) {
  const uint32_t r = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    put16(slot + 64 * r + 16 * (i ^ (r >> 1 & 3)), pack_bf16(x[8 * i], x[8 * i + 1]),
          pack_bf16(x[8 * i + 2], x[8 * i + 3]), pack_bf16(x[8 * i + 4], x[8 * i + 5]),
          pack_bf16(x[8 * i + 6], x[8 * i + 7]));
}
__device__ __forceinline__ void put_bytes(uint32_t slot, const uint32_t (&w)[8]) {
  const uint32_t r = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    put16(slot + 32 * r + 16 * (i ^ (r >> 2 & 1)), w[4 * i], w[4 * i + 1], w[4 * i + 2],
          w[4 * i + 3]);
}

// ---------------------------------------------------------------- forward
struct GatedOut {
  int M, F;
  int act;
  void* H;
  int64_t ldh;
  bool h_fp32, h_vec;
  int keep;
  void* kept;            // [M, 2, Fp] FP32 or int8
  uint8_t* exponents;    // [M, 2, Fp / 32]
  int Fp;                // 32 ceil(F / 32)
};

// One projection's 32 columns from column f of rows r0 .. r0 + 31, kept (plane 0: g, 1: u).
template <bool kSlots>
__device__ __forceinline__ void keep_run(const GatedOut& o, const CUtensorMap* map,
                                         StoreSlots& slots, int r0, int f, int plane,
                                         const uint32_t (&z)[32]) {
  const int row = r0 + (threadIdx.x & 31);
  const bool in = row < o.M;
  if (!RLK_STORE_OK(f + 32 <= o.Fp, &g_err_gated_linear)) return;
  const int64_t at = ((int64_t)row * 2 + plane) * o.Fp + f;
  if (o.keep == RLK_KEEP_FP32) {
    if constexpr (kSlots) {
      put_fp32(slots.take<true>(), z);
      slots.send(map, plane * o.Fp + f, r0);
    } else if (in) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(o.kept) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = make_uint4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
    }
    return;
  }
  float m[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    m[i] = max_magnitude(__uint_as_float(z[i]), __uint_as_float(z[i + 16]));
#pragma unroll
  for (int s = 8; s >= 1; s >>= 1)
#pragma unroll
    for (int i = 0; i < s; ++i) m[i] = max_magnitude(m[i], m[i + s]);
  const uint32_t e = int8_exponent(m[0]);
  const float inverse = int8_inverse(e);
  uint32_t w[8];
  const auto words = [&](bool hold) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x[4] = {__uint_as_float(z[4 * i]), __uint_as_float(z[4 * i + 1]),
                          __uint_as_float(z[4 * i + 2]), __uint_as_float(z[4 * i + 3])};
      w[i] = int8_word(x, inverse, hold);
    }
  };
  if (int8_holds(m[0], inverse))
    words(true);
  else
    words(false);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e == 255u) w[i] = 0u;
  if constexpr (kSlots) {
    put_bytes(slots.take<false>(), w);
    slots.send(map, plane * o.Fp + f, r0);
  } else if (in) {
    uint4* d = reinterpret_cast<uint4*>(static_cast<int8_t*>(o.kept) + at);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  if (in) o.exponents[at / kInt8Block] = (uint8_t)e;
}

template <int kAct>
__device__ __forceinline__ void value_run(const uint32_t (&g)[32], const uint32_t (&u)[32],
                                          float (&h)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    h[i] = gate_value<kAct>(__uint_as_float(g[i])) * __uint_as_float(u[i]);
}

// A tile's epilogue in one warp: accumulator columns [0, kCols) hold g and [kCols, 2 kCols) u of
// columns f0 .. f0 + kCols - 1 of the warp's rows r0 .. r0 + 31, of which it takes half `half`.
// kSlots: the warp has store slots.
template <int kCols, bool kSlots>
__device__ __forceinline__ void gated_tile(const GatedOut& o, const CUtensorMap* tm_h,
                                           const CUtensorMap* tm_kept, StoreSlots& slots,
                                           uint32_t taddr, int r0, int f0, int half) {
  if (r0 >= o.M) return;                    // uniform: depends on the warp's rows only
  constexpr int kChunks = kCols / 32, kMine = (kChunks + 1) / 2;
  const int end = half == 0 ? kMine : kChunks;
#pragma unroll 1
  for (int c = half * kMine; c < end; ++c) {
    const int f = f0 + 32 * c;
    if (f >= o.F) break;                    // uniform: depends on the tile only
    uint32_t g[32], u[32];
    __syncwarp();
    tmem_ld32(taddr + 32 * c, g);
    tmem_ld32(taddr + kCols + 32 * c, u);
    tmem_wait_ld();
    float h[32];
    if (o.act == RLK_ACT_SILU)
      value_run<RLK_ACT_SILU>(g, u, h);
    else
      value_run<RLK_ACT_GELU_TANH>(g, u, h);
    const int n = min(32, o.F - f);
    if (RLK_STORE_OK(f + n <= o.ldh, &g_err_gated_linear)) {
      if (kSlots && o.h_vec && n == 32) {
        if (o.h_fp32) {
          const uint32_t slot = slots.take<true>();
          uint32_t bits[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) bits[i] = __float_as_uint(h[i]);
          put_fp32(slot, bits);
        } else {
          put_bf16(slots.take<false>(), h);
        }
        slots.send(tm_h, f, r0);
      } else if (o.h_fp32) {
        store_block<true>(o.H, o.ldh, r0, o.M, f, n, !kSlots && o.h_vec, h);
      } else {
        store_block<false>(o.H, o.ldh, r0, o.M, f, n, !kSlots && o.h_vec, h);
      }
    }
    if (o.keep != RLK_KEEP_NONE) {
      // Columns past F are kept as 0: the products there are 0 times X, NaN where X is not finite.
      if (n < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= n) g[i] = u[i] = 0u;
      }
      keep_run<kSlots>(o, tm_kept, slots, r0, f, 0, g);
      keep_run<kSlots>(o, tm_kept, slots, r0, f, 1, u);
    }
  }
}

// More than 128 rows.  Bound by the tensor cores: 4096 x 4096 -> 16384 545 us by itself (2.02
// PFLOP/s, 1.05 of the measured product; 616 - 640 back to back, at the clock that the power cap
// leaves), 593 - 606 with FP32 projections kept, 568 with 8 bits.  The epilogue takes 3.4 us a
// tile (5.0 and 5.5 with them kept); at that rate a tile's MMAs take as long from K of about 690,
// 1010 and 1120 on.  Below, the epilogue bounds the call, and for some way above neither hides the
// other wholly: 4096 x K -> 16384 with K = 512 / 704 / 1024 / 1408 takes 109 / 125 / 160 / 204 us,
// 169 / 188 / 217 / 261 with FP32 kept, 161 / 170 / 188 / 233 with 8 bits, where the products
// alone at the measured rate are 72 / 98 / 143 / 197.
template <int kK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGatedThreads, 1)
    gated_linear_kernel(const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ CUtensorMap tm_h,
                        const __grid_constant__ CUtensorMap tm_kept, GatedSched sc, GatedOut o) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  const uint32_t tmem = pipe_setup<kEpilogueWarps>(ps);
  using TA = OperandTile<false, kHalfRows, kK>;
  using TB = GateUpHalf<kK>;
  using R = GatedRing<kK>;
  if (warp == 0) {
    if (lane == 0)
      producer_role<TA, TB, GatedSched, R>(&tm_x, &tm_w, sc, ps, &g_err_gated_linear);
    if (lane == 1 && ps.rank == 0) scheduler_role(sc, ps, &g_err_gated_linear);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && ps.rank == 0)
      mma_role<TA, TB, GatedSched, R>(sc, ps, tmem, idesc_bf16_f32(kPairRows, kBN, false, false),
                                      &g_err_gated_linear);
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;     // rows 32 q on, half of the columns
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    StoreSlots slots(R::reserve(ps.stages) + (warp - 2) * kSlotBytes);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int k = 0;; ++k) {
      const int u = warp_unit_take(sc, ps, k, &g_err_gated_linear);
      if (u < 0) break;
      if (!epilogue_acquire(ps, acc, acc_phase, &g_err_gated_linear)) break;
      int r0, b0;
      sc.tile_coords(u, 0, r0, b0);
      gated_tile<kGateCols, true>(o, &tm_h, &tm_kept, slots, tmem + acc * kAccCols + lane_off,
                                  r0 + (int)ps.rank * kHalfRows + q * 32, b0 / 2, half);
      epilogue_release(ps, acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    slots.finish();
  }
  pipe_teardown(tmem);
}

// At most 128 rows: the weight is streamed once, a CTA to a tile of kCols columns (solo_cols).
// Bound by HBM: 1 x 4096 -> 16384 43 us a call, 0.92 of the measured copy; with few tiles by a
// CTA's own stream and what comes before and after it (17 x 2048 -> 5461 17 us with a cold L2, 45
// MB).
template <int kARows, int kCols>
__global__ void __launch_bounds__(kGatedThreads, 1)
    gated_linear_solo_kernel(const __grid_constant__ CUtensorMap tm_x,
                             const __grid_constant__ CUtensorMap tm_w, GatedSched sc, GatedOut o) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  const uint32_t tmem = solo_setup<kEpilogueWarps>(ps);
  using R = SoloRing<kARows, 2 * kCols>;
  using TA = OperandTile<false, kARows>;
  using TB = GateUpBoth<kCols>;
  if (warp == 0) {
    if (lane == 0) solo_producer<TA, TB, R>(&tm_x, &tm_w, sc, ps, &g_err_gated_linear);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0)
      solo_mma<TA, TB, R>(sc, ps, tmem, idesc_bf16_f32(kHalfRows, 2 * kCols, false, false),
                          &g_err_gated_linear);
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;     // rows 32 q on, half of the columns
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    StoreSlots slots(0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int k = 0;; ++k) {
      const int u = solo_unit(sc, k);
      if (u < 0) break;
      if (!epilogue_acquire(ps, acc, acc_phase, &g_err_gated_linear)) break;
      int r0, b0;
      sc.tile_coords(u, 0, r0, b0);
      gated_tile<kCols, false>(o, nullptr, nullptr, slots, tmem + acc * kAccCols + lane_off, q * 32,
                               b0 / 2, half);
      solo_release(ps, acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  solo_teardown(tmem);
}

// ---------------------------------------------------------------- backward: G
struct GradOut {
  int M, F;
  int act;
  const void* dH;
  int64_t lddh;
  bool dh_fp32, dh_vec;
  uint16_t* G;           // [M, ldG] BF16: dL/dg in columns [0, F), dL/du in [F, 2 F)
  int64_t ldG;
  bool up_vec;           // column F of every row is on 16 bytes
};

template <int kAct>
__device__ __forceinline__ void slope_run(float (&d)[32], const uint32_t (&g)[32],
                                          const uint32_t (&u)[32], float (&dg)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float value, slope;
    gate_slope<kAct>(__uint_as_float(g[i]), value, slope);
    dg[i] = d[i] * __uint_as_float(u[i]) * slope;
    d[i] *= value;
  }
}

// G from projections formed again: the forward's loop, with another epilogue.  It takes 6.5 us a
// tile (dH is read when its chunk's turn comes), as long as the MMAs at K of about 1320: 4096 x K
// -> 16384 with K = 64 / 1024 / 1408 / 2048 takes 175 / 198 / 233 / 308 us, the products alone 9 /
// 143 / 197 / 286.
template <int kK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGatedThreads, 1)
    gated_grad_kernel(const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_gate,
                      const __grid_constant__ CUtensorMap tm_up, GatedSched sc, GradOut o) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  const uint32_t tmem = pipe_setup<kEpilogueWarps>(ps);
  using TA = OperandTile<false, kHalfRows, kK>;
  using TB = GateUpHalf<kK>;
  using R = GatedRing<kK>;
  if (warp == 0) {
    if (lane == 0)
      producer_role<TA, TB, GatedSched, R>(&tm_x, &tm_w, sc, ps, &g_err_gated_linear);
    if (lane == 1 && ps.rank == 0) scheduler_role(sc, ps, &g_err_gated_linear);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && ps.rank == 0)
      mma_role<TA, TB, GatedSched, R>(sc, ps, tmem, idesc_bf16_f32(kPairRows, kBN, false, false),
                                      &g_err_gated_linear);
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;     // rows 32 q on, half of the columns
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    StoreSlots slots(R::reserve(ps.stages) + (warp - 2) * kSlotBytes);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int k = 0;; ++k) {
      const int unit = warp_unit_take(sc, ps, k, &g_err_gated_linear);
      if (unit < 0) break;
      if (!epilogue_acquire(ps, acc, acc_phase, &g_err_gated_linear)) break;
      int r0, b0;
      sc.tile_coords(unit, 0, r0, b0);
      const int row0 = r0 + (int)ps.rank * kHalfRows + q * 32;
      const int f0 = b0 / 2;
      const uint32_t taddr = tmem + acc * kAccCols + lane_off;
#pragma unroll 1
      for (int c = half * (kGateCols / 64); c < (half + 1) * (kGateCols / 64); ++c) {
        const int f = f0 + 32 * c;
        if (f >= o.F || row0 >= o.M) break;     // uniform: depends on the tile and the warp only
        const int n = min(32, o.F - f);
        float d[32], dg[32];
        if (o.dh_fp32)
          load_block<true>(o.dH, o.lddh, row0, o.M, f, n, o.dh_vec, d);
        else
          load_block<false>(o.dH, o.lddh, row0, o.M, f, n, o.dh_vec, d);
        uint32_t g[32], u[32];
        __syncwarp();
        tmem_ld32(taddr + 32 * c, g);
        tmem_ld32(taddr + kGateCols + 32 * c, u);
        tmem_wait_ld();
        if (o.act == RLK_ACT_SILU)
          slope_run<RLK_ACT_SILU>(d, g, u, dg);
        else
          slope_run<RLK_ACT_GELU_TANH>(d, g, u, dg);
        if (!RLK_STORE_OK(o.F + f + n <= o.ldG, &g_err_gated_linear)) continue;
        if (n == 32) {
          put_bf16(slots.take<false>(), dg);
          slots.send(&tm_gate, f, row0);
        } else {
          store_block<false>(o.G, o.ldG, row0, o.M, f, n, false, dg);
        }
        if (o.up_vec && n == 32) {
          put_bf16(slots.take<false>(), d);
          slots.send(&tm_up, f, row0);
        } else {
          store_block<false>(o.G + o.F, o.ldG, row0, o.M, f, n, false, d);
        }
      }
      epilogue_release(ps, acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    slots.finish();
  }
  pipe_teardown(tmem);
}

// G from kept projections, eight columns a thread: one pass over 14 bytes a column in FP32, 8 in 8
// bits, bound by HBM: 4096 x 16384 from FP32 131 - 135 us (7.0 TB/s), 2000 x 5464 from 8 bits 19 -
// 21.  kVec: dH and both halves of G's rows allow 16-byte vectors; else they pass through shared
// memory (RowStage): 2000 x 5461 39 us, 50 with single elements for all operands.
template <bool kInt8, bool kDFp32, int kAct, bool kVec>
__global__ void __launch_bounds__(kRowThreads)
    gated_grad_kept_kernel(const void* __restrict__ kept, const uint8_t* __restrict__ exponents,
                           int Fp, GradOut o, RowLanes<8> lanes) {
  __shared__ __align__(16) float staged[kVec ? 1 : kRowThreads / 32][256];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * lanes.rows() + lanes.row();
  const bool in = row < o.M && RLK_STORE_OK(2 * (int64_t)o.F <= o.ldG, &g_err_gated_linear);
  const int64_t at = row * 2 * Fp;         // plane 0 of this row's kept projections
  const int64_t to = row * o.ldG;
  for (int f0 = (int)blockIdx.y * lanes.step(); f0 < o.F; f0 += (int)gridDim.y * lanes.step()) {
    const int f = f0 + lanes.col();
    float d[8], g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = g[i] = u[i] = 0.f;
    if constexpr (kVec) {
      if (in) load8<kDFp32, 8>(o.dH, row * o.lddh, f, 0, o.F, d);
    } else {
      RowStage(staged).load<kDFp32>(o.dH, row * o.lddh, f, o.F, in, d);
    }
    if (in && f < o.F) {
      if constexpr (kInt8) {
        const int8_t* q = static_cast<const int8_t*>(kept) + at;
        const uint8_t* e = exponents + at / kInt8Block;
        load_int8(q, e, f, g);
        load_int8(q + Fp, e + Fp / kInt8Block, f, u);
      } else {
        load8<true, 8>(kept, at, f, 0, Fp, g);
        load8<true, 8>(kept, at + Fp, f, 0, Fp, u);
      }
    }
    float dg[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float value, slope;
      gate_slope<kAct>(g[i], value, slope);
      dg[i] = d[i] * u[i] * slope;
      d[i] *= value;
    }
    if constexpr (kVec) {
      if (!in) continue;
      store8<false, 8>(o.G, to, f, 0, o.F, dg);
      store8<false, 8>(o.G, to + o.F, f, 0, o.F, d);
    } else {
      RowStage(staged).store<false>(o.G, to, f, o.F, in, dg);
      RowStage(staged).store<false>(o.G, to + o.F, f, o.F, in, d);
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxInner = (int64_t(1) << 30) - 256;
constexpr int64_t kMaxReduction = int64_t(1) << 20;
constexpr int64_t kUnitLimit = int64_t(1) << 31;

std::mutex g_attr_mutex;
bool g_attr_set[64];

template <class Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int kARows, int kCols>
constexpr int solo_smem() {
  return SoloRing<kARows, 2 * kCols>::kSmemBytes;
}
template <int kARows>
cudaError_t allow_solo() {
  cudaError_t e = allow_smem(gated_linear_solo_kernel<kARows, 128>, solo_smem<kARows, 128>());
  if (e == cudaSuccess)
    e = allow_smem(gated_linear_solo_kernel<kARows, 64>, solo_smem<kARows, 64>());
  if (e == cudaSuccess)
    e = allow_smem(gated_linear_solo_kernel<kARows, 32>, solo_smem<kARows, 32>());
  return e;
}

// Columns of g a tile of the one-CTA loop: 128, halved while twice the tiles still find an SM
// each, so that more of them stream the weight and a tile's epilogue, which ends the call, is
// shorter.  Measured (us, 128 / 64 / 32 columns, L2 written over before): 17 x 2048 -> 5461 22.5 /
// 18.5 / 26.6, 128 x 4096 -> 2000 32.8 / 26.6 / 24.6, 64 x 256 -> 1024 10.2 / 8.2 / 8.2, 1 x 4096
// -> 16384 60 / 65 / 80.  Past one wave of 128 columns, narrower tiles do no better (the step to a
// second round, at 19584, is there with either): 1 x 4096 -> 19456 (152 tiles) / 19584 / 22016 /
// 27648 / 28672 / 29568 with 128 columns 71 / 85 / 85 / 93 / 97 / 98, with 64 74 / 83 / 85 / 94 /
// 95 / 107; 100 rows 73 / 91 / 93 / 100 / 102 / 102 and 72 / 87 / 89 / 94 / 96 / 113.
int solo_cols(int64_t F, int64_t sms) {
  int w = 128;
  while (w > 32 && 2 * ceil_div(F, w) <= sms) w /= 2;
  return w;
}

template <int kARows>
cudaError_t launch_solo(int w, int grid, cudaStream_t s, const CUtensorMap& x,
                        const CUtensorMap& wm, const GatedSched& sc, const GatedOut& o) {
  return w == 128 ? launch_overlapped(gated_linear_solo_kernel<kARows, 128>, grid, kGatedThreads,
                                      solo_smem<kARows, 128>(), s, x, wm, sc, o)
         : w == 64 ? launch_overlapped(gated_linear_solo_kernel<kARows, 64>, grid, kGatedThreads,
                                       solo_smem<kARows, 64>(), s, x, wm, sc, o)
                   : launch_overlapped(gated_linear_solo_kernel<kARows, 32>, grid, kGatedThreads,
                                       solo_smem<kARows, 32>(), s, x, wm, sc, o);
}

cudaError_t ensure_attrs(int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_attr_set[dev]) return cudaSuccess;
  constexpr int kDeep = GatedRing<64>::kSmemBytes;
  constexpr int kWide = GatedRing<128>::kSmemBytes;
  cudaError_t e;
  if ((e = allow_smem(gated_linear_kernel<64>, kDeep)) != cudaSuccess ||
      (e = allow_smem(gated_linear_kernel<128>, kWide)) != cudaSuccess ||
      (e = allow_smem(gated_grad_kernel<64>, kDeep)) != cudaSuccess ||
      (e = allow_smem(gated_grad_kernel<128>, kWide)) != cudaSuccess ||
      (e = allow_solo<32>()) != cudaSuccess || (e = allow_solo<128>()) != cudaSuccess)
    return e;
  g_attr_set[dev] = true;
  return cudaSuccess;
}

rlk_status cuda_failed() {
  cudaGetLastError();
  return RLK_ERR_CUDA;
}

// [G (backward)][unit counter, 256 bytes][padded copy of X][padded copy of W], each region
// 256-byte aligned; copies only of operands that TMA cannot read in place.
struct GatedPlan {
  int64_t ldG = 0;
  bool stage_x = false, stage_w = false;
  int64_t ldx = 0, ldw = 0;
  size_t off_ctr = 0, off_x = 0, off_w = 0, total = 0;
};

rlk_status gated_plan(bool backward, const void* X, int64_t M, int64_t K, int64_t ldx,
                      const void* W, int64_t F, int64_t ldw, GatedPlan* p) {
  if (M < 0 || M >= kMaxExtent || K < 1 || K >= kMaxReduction || F < 1 || F >= kMaxInner ||
      ldx < K || ldw < K || ldx >= kPitchLimit || ldw >= kPitchLimit)
    return RLK_ERR_SHAPE;
  // work units are numbered in ints, here and in the backward's products (128-column tiles)
  const int64_t rb = ceil_div(M, kPairRows), kb = ceil_div(K, kBN / 2);
  if (rb * ceil_div(F, kGateCols) >= kUnitLimit || rb * kb >= kUnitLimit ||
      ceil_div(2 * F, kPairRows) * kb >= kUnitLimit)
    return RLK_ERR_SHAPE;
  p->ldG = ceil_div(2 * F, 8) * 8;
  p->stage_x = M > 0 && !tma_ready(X, ldx);
  p->stage_w = M > 0 && !tma_ready(W, ldw);
  p->ldx = p->stage_x ? staged_ld(K) : ldx;
  p->ldw = p->stage_w ? staged_ld(K) : ldw;
  size_t off = backward ? align_up((size_t)M * p->ldG * 2, 256) : 0;
  p->off_ctr = off;
  off += 256;
  p->off_x = off;
  if (p->stage_x) off = align_up(off + (size_t)M * p->ldx * 2, 256);
  p->off_w = off;
  if (p->stage_w) off = align_up(off + (size_t)(2 * F) * p->ldw * 2, 256);
  p->total = off;
  return RLK_OK;
}

// The operands as the kernels read them: in place, or the workspace's copies (made by stage()).
struct Operands {
  const void *x, *w;
};
Operands operands_of(const GatedPlan& p, const void* X, const void* W, uint8_t* ws) {
  return {p.stage_x ? ws + p.off_x : X, p.stage_w ? ws + p.off_w : W};
}
cudaError_t stage(const GatedPlan& p, bool x_used, bool w_used, const void* X, int64_t M, int64_t K,
                  int64_t ldx, const void* W, int64_t F, int64_t ldw, uint8_t* ws, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (x_used && p.stage_x)
    e = launch_stage_bf16(static_cast<const uint16_t*>(X), M, K, ldx,
                          reinterpret_cast<uint16_t*>(ws + p.off_x), p.ldx, s);
  if (e == cudaSuccess && w_used && p.stage_w)
    e = launch_stage_bf16(static_cast<const uint16_t*>(W), 2 * F, K, ldw,
                          reinterpret_cast<uint16_t*>(ws + p.off_w), p.ldw, s);
  return e;
}

bool encode_x(CUtensorMap* map, const GatedPlan& p, const void* x, int64_t M, int64_t K, int rows) {
  return encode_bf16_2d(map, x, K, M, p.ldx, kBK, rows);
}
bool encode_w(CUtensorMap* map, const GatedPlan& p, const void* w, int64_t K, int64_t F, int rows,
              int planes) {
  return encode_bf16_3d(map, w, K, F, 2, p.ldw, (uint64_t)F * p.ldw, kBK, rows, planes);
}

// The 2-SM loop's schedule; zeroes the unit counter where one is used.
cudaError_t pair_sched(int64_t M, int64_t K, int64_t F, int stage_k, int64_t clusters, int* counter,
                       cudaStream_t s, GatedSched* sc, int* grid) {
  sc->order.rows = (int)ceil_div(M, kPairRows);
  sc->order.cols = (int)ceil_div(F, kGateCols);
  sc->order.band = band_rows(sc->order.rows, K, kPairRows);
  sc->nkb = (int)ceil_div(K, stage_k);
  sc->nkb64 = (int)ceil_div(K, kBK);
  sc->tile_rows = kBN;
  sc->counter = nullptr;
  const int64_t units = (int64_t)sc->order.rows * sc->order.cols;
  *grid = 2 * (int)(units < clusters ? units : clusters);
  if (!ordered_units(units, clusters)) return cudaSuccess;
  sc->counter = counter;
  return cudaMemsetAsync(counter, 0, sizeof(int), s);
}

// Both products of a backward in one launch over both tile lists (the same bits), so that the one
// with the shorter reduction fills the SM pairs that the few tiles of the long one leave idle.
// Apart, the long one has narrow tiles, which take 0.69 of a wide tile's time, and its launch
// overlaps the other's ends; so one launch pays where the long one's 256 x 256 tiles fill at most
// half of the pairs, the other product takes about half as long as one of them or more, counting
// 64-wide reduction blocks and six more for a tile's store, and has eight tiles a pair or more to
// deal out. Measured (us for the whole backward from 8 bits, one launch / two; in brackets that
// ratio and the tiles a pair): grad X the longer, 255 x 4096 -> 11000 153 / 190 (0.53, 18), 37 x
// 6144 -> 4856 96 / 115 (0.55, 12), 100 x 9728 -> 2000 71 / 75 (1.02, 8.0), 500 x 4864 -> 2000 65
// / 57 (0.89, 4.0), 512 x 2048 -> 8192 125 / 112 (0.37, 6.7), 42 x 1544 -> 14080 175 / 151 (0.16,
// 10); grad W the longer, 22410 x 5120 -> 72 179 / 237 (0.59, 23), 27678 x 3840 -> 128 186 / 232
// (0.50, 21), 10000 x 4096 -> 128 91 / 97 (0.54, 8.4), 2500 x 9728 -> 64 54 / 51 (1.00, 5.0),
// 10000 x 2048 -> 512 105 / 88 (0.59, 4.2), 44416 x 1280 -> 80 260 / 221 (0.15, 11).
bool one_launch(int64_t M, int64_t K, int64_t F, int64_t pairs) {
  const int64_t red_long = M > 2 * F ? M : 2 * F, red_short = M > 2 * F ? 2 * F : M;
  const int64_t kb = ceil_div(K, kBN);
  const int64_t short_tiles = ceil_div(red_long, kPairRows) * kb;
  if (2 * ceil_div(red_short, kPairRows) * kb > pairs || short_tiles < 8 * pairs) return false;
  return 100 * short_tiles * (ceil_div(red_short, kBK) + 6) > 45 * pairs * ceil_div(red_long, kBK);
}

bool known_activation(int a) { return a == RLK_ACT_SILU || a == RLK_ACT_GELU_TANH; }

rlk_status check_kept(int keep, const void* kept, const uint8_t* exponents) {
  if (keep == RLK_KEEP_NONE) return RLK_OK;
  if (!kept || (keep == RLK_KEEP_INT8 && !exponents)) return RLK_ERR_NULL;
  return is_aligned(kept, 32) ? RLK_OK : RLK_ERR_ALIGN;
}

}  // namespace

uint32_t take_error_gated_linear() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_gated_linear, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaMemcpyToSymbol(g_err_gated_linear, &zero, sizeof zero);
  cudaGetLastError();
  return v;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

size_t rlk_gated_linear_workspace_size(const void* X, int64_t M, int64_t K, int64_t ldx,
                                       const void* W, int64_t F, int64_t ldw) {
  GatedPlan p;
  return gated_plan(false, X, M, K, ldx, W, F, ldw, &p) == RLK_OK ? p.total : 0;
}

rlk_status rlk_gated_linear(const void* X, int64_t M, int64_t K, int64_t ldx, const void* W,
                            int64_t F, int64_t ldw, int activation, void* H, int h_dtype,
                            int64_t ldh, int keep, void* kept, uint8_t* kept_exponents,
                            void* workspace, size_t workspace_bytes, void* stream) {
  RLK_CALL_RANGE();
  GatedPlan p;
  rlk_status st = gated_plan(false, X, M, K, ldx, W, F, ldw, &p);
  if (st != RLK_OK) return st;
  if (ldh < F || ldh >= kPitchLimit) return RLK_ERR_SHAPE;
  if (!known_dtype(h_dtype)) return RLK_ERR_DTYPE;
  if (!known_activation(activation) || keep < RLK_KEEP_NONE || keep > RLK_KEEP_INT8)
    return RLK_ERR_VALUE;
  if (M == 0) return RLK_OK;
  if (!X || !W || !H) return RLK_ERR_NULL;
  if (!is_aligned(X, 2) || !is_aligned(W, 2) || !is_aligned(H, dtype_bytes(h_dtype)))
    return RLK_ERR_ALIGN;
  if ((st = check_kept(keep, kept, kept_exponents)) != RLK_OK) return st;
  if (!workspace || !is_aligned(workspace, 256) || workspace_bytes < p.total)
    return RLK_ERR_WORKSPACE;
  DeviceInfo dev;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  if (ensure_attrs(dev.device) != cudaSuccess) return cuda_failed();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Operands in = operands_of(p, X, W, ws);
  const bool solo = M <= kHalfRows;
  const int x_rows = M <= 32 ? 32 : kHalfRows;
  const int cols = solo ? solo_cols(F, dev.sm_count) : kGateCols;      // a tile's, of g
  CUtensorMap tm_x, tm_w;
  if (!encode_x(&tm_x, p, in.x, M, K, x_rows) ||
      !encode_w(&tm_w, p, in.w, K, F, cols, solo ? 2 : 1))
    return RLK_ERR_CUDA;
  GatedOut o;
  o.M = (int)M;
  o.F = (int)F;
  o.act = activation;
  o.H = H;
  o.ldh = ldh;
  o.h_fp32 = h_dtype == RLK_FP32;
  o.h_vec = block_vec(H, ldh, dtype_bytes(h_dtype));
  o.keep = keep;
  o.kept = kept;
  o.exponents = kept_exponents;
  o.Fp = (int)(ceil_div(F, kInt8Block) * kInt8Block);
  // the maps of what the 2-SM loop stores by TMA (see StoreSlots)
  CUtensorMap tm_h = {}, tm_kept = {};
  if (!solo &&
      ((o.h_vec && !encode_store_2d(&tm_h, H, dtype_bytes(h_dtype), F, M, ldh)) ||
       (keep != RLK_KEEP_NONE && !encode_store_2d(&tm_kept, kept, keep == RLK_KEEP_FP32 ? 4 : 1,
                                                  2 * (uint64_t)o.Fp, M, 2 * (uint64_t)o.Fp))))
    return RLK_ERR_CUDA;
  if (stage(p, true, true, X, M, K, ldx, W, F, ldw, ws, s) != cudaSuccess) return cuda_failed();
  GatedSched sc;
  cudaError_t e;
  if (solo) {
    sc.order.rows = 1;
    sc.order.cols = (int)ceil_div(F, cols);
    sc.order.band = 1;
    sc.counter = nullptr;
    sc.nkb = sc.nkb64 = (int)ceil_div(K, kBK);
    sc.tile_rows = 2 * cols;
    const int grid = sc.order.cols < dev.sm_count ? sc.order.cols : dev.sm_count;
    e = x_rows == 32 ? launch_solo<32>(cols, grid, s, tm_x, tm_w, sc, o)
                     : launch_solo<128>(cols, grid, s, tm_x, tm_w, sc, o);
  } else {
    const int stage_k = M > kWideStageRows ? 128 : 64;
    int grid;
    e = pair_sched(M, K, F, stage_k, dev.sm_count / 2, reinterpret_cast<int*>(ws + p.off_ctr), s,
                   &sc, &grid);
    if (e == cudaSuccess)
      e = stage_k == 128 ? launch_overlapped(gated_linear_kernel<128>, grid, kGatedThreads,
                                             GatedRing<128>::kSmemBytes, s, tm_x, tm_w, tm_h,
                                             tm_kept, sc, o)
                         : launch_overlapped(gated_linear_kernel<64>, grid, kGatedThreads,
                                             GatedRing<64>::kSmemBytes, s, tm_x, tm_w, tm_h,
                                             tm_kept, sc, o);
  }
  return e == cudaSuccess ? RLK_OK : cuda_failed();
}

size_t rlk_gated_linear_backward_workspace_size(const void* X, int64_t M, int64_t K, int64_t ldx,
                                                const void* W, int64_t F, int64_t ldw) {
  GatedPlan p;
  return gated_plan(true, X, M, K, ldx, W, F, ldw, &p) == RLK_OK ? p.total : 0;
}

rlk_status rlk_gated_linear_backward(const void* dH, int dh_dtype, int64_t M, int64_t F,
                                     int64_t lddh, const void* X, int64_t K, int64_t ldx,
                                     const void* W, int64_t ldw, int activation, int keep,
                                     const void* kept, const uint8_t* kept_exponents, void* dX,
                                     int dx_dtype, int64_t lddx, void* dW, int dw_dtype,
                                     int64_t lddw, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  RLK_CALL_RANGE();
  // ---- every check, including those of the products below, before the first launch
  GatedPlan p;
  rlk_status st = gated_plan(true, X, M, K, ldx, W, F, ldw, &p);
  if (st != RLK_OK) return st;
  if (lddh < F || lddh >= kPitchLimit || (dX && (lddx < K || lddx >= kPitchLimit)) ||
      (dW && (lddw < K || lddw >= kPitchLimit)))
    return RLK_ERR_SHAPE;
  if (!known_dtype(dh_dtype) || (dX && !known_dtype(dx_dtype)) || (dW && !known_dtype(dw_dtype)))
    return RLK_ERR_DTYPE;
  if (!known_activation(activation) || keep < RLK_KEEP_NONE || keep > RLK_KEEP_INT8)
    return RLK_ERR_VALUE;
  if (!dX && !dW) return RLK_OK;
  if ((dX && !is_aligned(dX, dtype_bytes(dx_dtype))) ||
      (dW && !is_aligned(dW, dtype_bytes(dw_dtype))))
    return RLK_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (M == 0) {
    if (!dW) return RLK_OK;
    if ((st = device_ready(&dev)) != RLK_OK) return st;
    const size_t es = dtype_bytes(dw_dtype);
    return cudaMemset2DAsync(dW, lddw * es, 0, K * es, 2 * F, s) == cudaSuccess ? RLK_OK
                                                                                : cuda_failed();
  }
  const bool x_used = dW || keep == RLK_KEEP_NONE, w_used = dX || keep == RLK_KEEP_NONE;
  if (!dH || (x_used && !X) || (w_used && !W)) return RLK_ERR_NULL;
  if (!is_aligned(dH, dtype_bytes(dh_dtype)) || !is_aligned(X, 2) || !is_aligned(W, 2))
    return RLK_ERR_ALIGN;
  if ((st = check_kept(keep, kept, kept_exponents)) != RLK_OK) return st;
  if (!workspace || !is_aligned(workspace, 256) || workspace_bytes < p.total)
    return RLK_ERR_WORKSPACE;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  if (ensure_attrs(dev.device) != cudaSuccess) return cuda_failed();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Operands in = operands_of(p, X, W, ws);
  uint16_t* G = reinterpret_cast<uint16_t*>(ws);
  const bool up_vec = block_vec(G + F, p.ldG, 2);
  CUtensorMap tm_x, tm_w, tm_gate = {}, tm_up = {};
  if (keep == RLK_KEEP_NONE && (!encode_x(&tm_x, p, in.x, M, K, kHalfRows) ||
                                !encode_w(&tm_w, p, in.w, K, F, kGateCols, 1) ||
                                !encode_store_2d(&tm_gate, G, 2, F, M, p.ldG) ||
                                (up_vec && !encode_store_2d(&tm_up, G + F, 2, F, M, p.ldG))))
    return RLK_ERR_CUDA;
  if (stage(p, x_used, w_used, X, M, K, ldx, W, F, ldw, ws, s) != cudaSuccess) return cuda_failed();

  GradOut o;
  o.M = (int)M;
  o.F = (int)F;
  o.act = activation;
  o.dH = dH;
  o.lddh = lddh;
  o.dh_fp32 = dh_dtype == RLK_FP32;
  o.dh_vec = block_vec(dH, lddh, dtype_bytes(dh_dtype));
  o.G = G;
  o.ldG = p.ldG;
  o.up_vec = up_vec;
  int* counter = reinterpret_cast<int*>(ws + p.off_ctr);
  cudaError_t e;
  if (keep == RLK_KEEP_NONE) {
    const int stage_k = M > kWideStageRows ? 128 : 64;
    GatedSched sc;
    int grid;
    e = pair_sched(M, K, F, stage_k, dev.sm_count / 2, counter, s, &sc, &grid);
    if (e == cudaSuccess)
      e = stage_k == 128 ? launch_overlapped(gated_grad_kernel<128>, grid, kGatedThreads,
                                             GatedRing<128>::kSmemBytes, s, tm_x, tm_w, tm_gate,
                                             tm_up, sc, o)
                         : launch_overlapped(gated_grad_kernel<64>, grid, kGatedThreads,
                                             GatedRing<64>::kSmemBytes, s, tm_x, tm_w, tm_gate,
                                             tm_up, sc, o);
  } else {
    const int Fp = (int)(ceil_div(F, kInt8Block) * kInt8Block);
    const auto launch = [&](auto q8, auto d32, auto v) {
      constexpr bool kQ = decltype(q8)::value, kD = decltype(d32)::value;
      constexpr bool kVec = decltype(v)::value;
      const RowLanes<8> lanes = row_lanes<8>(F, kVec ? 2 : 5);
      const int64_t steps = ceil_div(F, lanes.step());
      const dim3 grid((unsigned)ceil_div(M, lanes.rows()),
                      (unsigned)(steps < 65535 ? steps : 65535));
      return activation == RLK_ACT_SILU
                 ? launch_overlapped(gated_grad_kept_kernel<kQ, kD, RLK_ACT_SILU, kVec>, grid,
                                     kRowThreads, 0, s, kept, kept_exponents, Fp, o, lanes)
                 : launch_overlapped(gated_grad_kept_kernel<kQ, kD, RLK_ACT_GELU_TANH, kVec>, grid,
                                     kRowThreads, 0, s, kept, kept_exponents, Fp, o, lanes);
    };
    const bool vec = o.dh_vec && o.up_vec && F % 8 == 0;
    e = by_dtypes(keep == RLK_KEEP_INT8 ? RLK_FP32 : RLK_BF16, dh_dtype, [&](auto q8, auto d32) {
      return vec ? launch(q8, d32, Const<true>()) : launch(q8, d32, Const<false>());
    });
  }
  if (e != cudaSuccess) return cuda_failed();
  // The products read G and the (possibly copied) operands, all TMA-ready: the counter is all the
  // workspace they need, and every argument that they check was checked above.
  if (dX && dW && one_launch(M, K, F, dev.sm_count / 2))
    return launch_fwd_and_db(o.G, M, 2 * F, p.ldG, in.w, K, p.ldw, dX, dx_dtype, lddx, in.x, p.ldx,
                             dW, dw_dtype, lddw, counter, s);
  return rlk_det_linear_backward(o.G, RLK_BF16, M, 2 * F, p.ldG, in.x, K, p.ldx, in.w, p.ldw, dX,
                                 dx_dtype, dX ? lddx : K, dW, dw_dtype, dW ? lddw : K,
                                 ws + p.off_ctr, 256, stream);
}

}  // extern "C"
