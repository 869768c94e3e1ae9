// What the kernels that run over vocabulary splits share: the work order, and one
// row's logits 32 columns at a time as their epilogues handle them (bias and
// vocabulary-tail mask, one column out of the 32, the online maximum m and sum of
// exponentials s with their fixed-order merge).  Every operation is rounded
// explicitly, so all kernels that fold the same logits get the same (m, s) bits.
#pragma once

#include <float.h>
#include <math.h>

#include "rlk_device.cuh"

namespace rlk {

// Units = (vocabulary split, row block).
struct VocabSched {
  Banded order;    // rows = 256-row blocks, cols = this call's vocabulary splits
  int* counter;    // zeroed unit counter in the workspace (units in order), or null (round-robin)
  int S;           // vocabulary splits in this call (all S, or a shard's run of them)
  int vps;         // 256-id tiles per split
  int vtiles;      // 256-id tiles of the weight rows this call reads
  int tile0;       // global index of the first of those tiles (0 unless a vocabulary shard)
  int nkb;         // reduction stages over H (64 or 128 wide)
  int nkb64;       // 64-wide blocks of H
  __device__ __forceinline__ int num_units() const { return order.count(); }
  __device__ __forceinline__ int split_of(int u) const {
    int rb, j;
    order.unit(u, rb, j);
    return j;
  }
  __device__ __forceinline__ int rb_of(int u) const {
    int rb, j;
    order.unit(u, rb, j);
    return rb;
  }
  __device__ __forceinline__ int first_tile(int u) const { return split_of(u) * vps; }
  __device__ __forceinline__ int unit_tiles(int u) const {
    const int t0 = first_tile(u);
    return min(vps, vtiles - t0);
  }
  int rows_per_unit;   // 256 (a CTA pair's rows) or 128 (one CTA's, the one-CTA loop)
  __device__ __forceinline__ void tile_coords(int u, int i, int& a0, int& b0) const {
    a0 = rb_of(u) * rows_per_unit;
    b0 = (first_tile(u) + i) * kBN;
  }
};

// z = the chunk's accumulators plus bias, -inf at and past vocabulary id V.  Column
// i's bias comes from the warp's BiasTile (a shuffle: every lane takes part).
__device__ __forceinline__ void chunk_logits(const uint32_t (&r)[32], int vbase, int V,
                                             bool has_bias, const BiasTile& bias, int c,
                                             float (&z)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(r[i]);
  if (has_bias) {
    if (vbase + 32 <= V) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        z[i] = __fadd_rn(z[i], bias_tile_at(bias, c, i));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float b = bias_tile_at(bias, c, i);
        if (vbase + i < V) z[i] = __fadd_rn(z[i], b);
      }
    }
  }
  if (vbase + 32 > V) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (vbase + i >= V) z[i] = -INFINITY;
  }
}

// z[di] (0 <= di < 32) through a fixed 5-level select tree (keeps z in registers).
__device__ __forceinline__ float chunk_at(const float (&z)[32], int di) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = (di & 16) ? z[i + 16] : z[i];
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) t[i] = (di & w) ? t[i + w] : t[i];
  return t[0];
}

// Folds the chunk into (m, s) with s = sum 2^((z - m) * scale); scale = log2(e), or
// log2(e) / T for logits at temperature T.  z - m is formed first, so the running
// maximum's own term is exactly 2^0 = 1: s >= 1 once a logit was above -inf.  m is at
// least the lowest finite number: a chunk of banned logits (bias -inf) adds 2^-inf = 0
// each where -inf - -inf would be NaN, and a NaN logit reaches s below a finite m, so
// that the merge does not take the split for an empty one.
__device__ __forceinline__ void chunk_fold(const float (&z)[32], float scale, float& m, float& s) {
  // chunk maximum (fixed pairwise tree)
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = fmaxf(z[2 * i], z[2 * i + 1]);
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) t[i] = fmaxf(t[i], t[i + w]);
  const float mn = fmaxf(fmaxf(m, t[0]), -FLT_MAX);
  const float down = ex2_approx(__fmul_rn(__fsub_rn(m, mn), scale));   // m = -inf -> 0
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; ++i)
    a[i & 3] = __fadd_rn(a[i & 3], ex2_approx(__fmul_rn(__fsub_rn(z[i], mn), scale)));
  const float cs = __fadd_rn(__fadd_rn(a[0], a[1]), __fadd_rn(a[2], a[3]));
  s = __fadd_rn(__fmul_rn(s, down), cs);
  m = mn;
}

// (m, s) pair merge with explicit roundings, so merge(a, b) == merge(b, a) bitwise.
__device__ __forceinline__ void merge_ms(float& M, float& s, float m2, float s2,
                                         float scale = kLog2e) {
  if (m2 == -INFINITY) return;
  if (M == -INFINITY) {
    M = m2;
    s = s2;
    return;
  }
  const float Mn = fmaxf(M, m2);
  const float e1 = ex2_approx(__fmul_rn(__fsub_rn(M, Mn), scale));
  const float e2 = ex2_approx(__fmul_rn(__fsub_rn(m2, Mn), scale));
  s = __fadd_rn(__fmul_rn(s, e1), __fmul_rn(s2, e2));
  M = Mn;
}

}  // namespace rlk
