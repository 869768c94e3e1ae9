// Distillation of a linear student from a teacher's top logits, on sm_103a.
//
// Row r has K slots (id_k, t_k): vocabulary ids with the teacher's logits there.  A
// slot whose id is outside [0, V) or whose logit is -inf is empty (lists of unequal
// length are padded with id -1).  At temperature T, over the row's used slots,
//   log q_k = t_k / T - L,  L = teacher_lse[r], or log sum_k exp(t_k / T) if not given
//   z[r, v] = hidden[r] . W[v] (+ bias[v]),   lse[r] = log sum_v exp(z[r, v] / T)
//   loss[r] = T^2 sum_k q_k (log q_k - z[r, id_k] / T + lse[r])
// and, with g[r] = dL/dloss[r],
//   G[r, v] = dL/dz[r, v] = g[r] T (Q exp(z[r, v] / T - lse[r]) - sum_{k: id_k = v} q_k)
//   grad_hidden = G . W,  grad_weight = G^T . hidden,  grad_bias = sum_r G.
// A row without used slots has loss 0 and gradient 0.
//
// The work is the product hidden . W^T (2 N H V operations, tensor cores); everything
// else rides along so that the [N, V] logits need not exist:
//  * distill_lists_kernel (one block per row): q and its sums, the used slots sorted by id
//    (rank by counting: K^2 compares over the block, and a stable order whatever the
//    lists hold), and where each vocabulary split's ids start.
//  * distill_partials_kernel / distill_solo_kernel: the tcgen05 loops of the fused
//    linear-logp (2-SM pairs; one CTA for at most 128 rows).  The epilogue thread that
//    owns a row folds (m, s) as there and walks the row's sorted ids alongside the
//    columns: an id costs one compare per 32 columns and, when hit, one select tree,
//    so D = sum q z is gathered from the accumulators and no row of W is read twice.
//  * distill_combine_kernel: the fixed-order merge over the splits, and the loss.
//  * distill_grad_kernel: the same loop again; the epilogue forms G in FP32, takes the
//    32-row column sums for grad_bias from it, and stores it rounded to BF16, the type
//    in which the two products (det_gemm) read it.
//  * distill_grad_logits_kernel: the same G, bit for bit, from logits that the forward kept
//    (4 N V bytes): one pass at memory speed in place of the product's 2 N H V operations.
//
// Sums are FP32 and every logit is the tensor core's FP32 sum over H, whose own error at
// H = 4096 is some 1e-6 of the logit: lse is within 6e-6 (relative, worst of 60 random calls at
// H = 2048 and 4096) of 64 bits.  The loss is a difference of parts as large as |z| T and
// T^2 log V, so its error is absolute: beside the logits' own, about 2e-7 T max|z| and 3e-7
// max(T^2 Q, loss), measured with exact logits.  At T = 1000 that is as large as the loss of a
// student close to the teacher, whatever the sums are joined in, so T ends at 100.  The one
// rounding to fewer bits is G's to BF16, the type the products' tensor instructions read: it
// raises the gradients' error against 64 bits (relative, root mean square) from the 0.0017 of
// their own BF16 rounding to 0.0024.  grad_bias is summed before it.
#include <limits.h>
#include <math.h>

#include <mutex>

#include <cuda_bf16.h>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_pipeline.cuh"
#include "rlk_solo.cuh"
#include "rlk_vocab.cuh"

namespace rlk {

__device__ unsigned int g_err_linear_distill = 0;

namespace {

constexpr int64_t kMaxSlots = 1024;
constexpr int64_t kLdLimit = int64_t(1) << 36;
constexpr int64_t kUnitLimit = int64_t(1) << 31;

// ---------------------------------------------------------------- teacher lists
// The teacher's lists as the epilogues read them: row r's used slots in ascending id
// order at [r * K], their number cut at span boundaries by first[r * (spans + 1) + j]
// (slots first[j] .. first[j + 1] - 1 have ids in span j), and two sums of the row: E and
// the norm of q for the forward, Q (second) for the backward.
struct Lists {
  int* ids;
  float* q;
  uint16_t* first;
  float2* sums;
  int K, spans;
  int64_t span;      // vocabulary ids per span
};

struct ListArgs {
  const int64_t* ids;
  int64_t ld_ids;
  const void* logits;
  int64_t ld_logits;
  int logits_fp32;
  const float* lse;       // the teacher's own log-sum-exp at this temperature, or null
  float temperature;
  double inv_t;
  int N, V;
  bool backward;
};

// Sum and maximum over the block in a fixed order: every thread's value through a xor
// butterfly in its warp, then the warps' results in ascending order.
template <bool kMax>
__device__ __forceinline__ float block_fold(float v, float* warp_out) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = kMax ? fmaxf(v, o) : __fadd_rn(v, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_out[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_out[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w)
    v = kMax ? fmaxf(v, warp_out[w]) : __fadd_rn(v, warp_out[w]);
  return v;
}

// Bound by latency: a row's K (id, logit) pairs are read once, and a chain of block-wide steps
// follows.  Counting ranks costs K^2 shared reads over 256 threads and no barriers: 12.6 us for
// 2048 rows of 64 slots (0.01 of the forward it precedes at H = 4096, V = 151936), 5.7 us for 1024
// rows of 20.  Long lists pay for the square: 2048 rows of 256 slots 44 us, of 1024 slots 560 us
// (0.3 of the 1.86 ms that this forward then takes, and once more in the backward).
__global__ void __launch_bounds__(256) distill_lists_kernel(ListArgs a, Lists out) {
  extern __shared__ int smem_lists[];
  int* key = smem_lists;                                    // [K] id, or INT_MAX when empty
  int* sorted = smem_lists + out.K;                         // [K]
  float* val = reinterpret_cast<float*>(sorted + out.K);    // [K] t, then q
  __shared__ float warp_out[8];
  __shared__ int used;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int row = blockIdx.x;
  const int K = out.K;
  float top = -INFINITY;
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const int64_t id = __ldg(a.ids + (int64_t)row * a.ld_ids + k);
    const int64_t at = (int64_t)row * a.ld_logits + k;
    const float t = a.logits_fp32
                        ? __ldg(static_cast<const float*>(a.logits) + at)
                        : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.logits) + at)
                                          << 16);
    const bool on = id >= 0 && id < a.V && t != -INFINITY;
    key[k] = on ? (int)id : INT_MAX;
    val[k] = on ? t : -INFINITY;
    top = fmaxf(top, val[k]);
  }
  if (threadIdx.x == 0) used = 0;
  // y = (t - top) / T <= 0 is small where T is large, and so keeps the digits that T^2 needs
  top = block_fold<true>(top, warp_out);
  float norm;                                      // q = exp(y) / norm
  if (a.lse) {
    // exp(lse - top / T), the exponent in two parts: rounded to one it would move every q by
    // 5e-7 of itself, and the loss with them
    const double x = __ldg(a.lse + row) - top * a.inv_t;
    const float near = (float)x;
    norm = __fmul_rn(expf(near), __fadd_rn(1.f, (float)(x - near)));
  } else {
    float s = 0.f;
    for (int k = threadIdx.x; k < K; k += blockDim.x)
      if (key[k] != INT_MAX)
        s = __fadd_rn(s, expf(__fdiv_rn(__fsub_rn(val[k], top), a.temperature)));
    norm = block_fold<false>(s, warp_out);
  }
  float e = 0.f, sum = 0.f;
  int n = 0;
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    float q = 0.f;
    if (key[k] != INT_MAX) {
      const float y = __fdiv_rn(__fsub_rn(val[k], top), a.temperature);
      q = __fdiv_rn(expf(y), norm);
      if (q > 0.f) e = __fadd_rn(e, __fmul_rn(q, y));
      sum = __fadd_rn(sum, q);
      ++n;
    }
    val[k] = q;
  }
  if (a.backward)
    sum = block_fold<false>(sum, warp_out);
  else
    e = block_fold<false>(e, warp_out);
  if (n) atomicAdd(&used, n);      // a whole number: its order does not matter
  __syncthreads();
  if (threadIdx.x == 0 && RLK_STORE_OK(row < a.N, &g_err_linear_distill))
    out.sums[row] = a.backward ? make_float2(0.f, sum) : make_float2(e, a.lse ? top : norm);
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const int id = key[k];
    int rank = 0;
    for (int j = 0; j < K; ++j) rank += key[j] < id || (key[j] == id && j < k);
    sorted[rank] = id;
    const int64_t at = (int64_t)row * K + rank;
    if (RLK_STORE_OK(rank < K && row < a.N, &g_err_linear_distill)) {
      out.ids[at] = id;
      out.q[at] = val[k];
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j <= out.spans; j += blockDim.x) {
    const int64_t bound = j * out.span;
    int lo = 0, hi = used;                       // first used slot with id >= bound
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < bound) lo = mid + 1;
      else hi = mid;
    }
    if (RLK_STORE_OK(row < a.N, &g_err_linear_distill))
      out.first[(int64_t)row * (out.spans + 1) + j] = (uint16_t)lo;
  }
}

// A row's walk along its sorted slots: the next id (INT_MAX past the span) and its q.
struct SlotWalk {
  const int* ids;
  const float* q;
  int at, end;
  int id;
  float w;
  __device__ __forceinline__ void load() {
    id = INT_MAX;
    if (at < end) {
      id = __ldg(ids + at);
      w = __ldg(q + at);
    }
  }
  __device__ __forceinline__ void start(const Lists& l, int row, int span, bool valid) {
    at = end = 0;
    w = 0.f;
    if (valid) {
      const uint16_t* f = l.first + (int64_t)row * (l.spans + 1) + span;
      at = __ldg(f);
      end = __ldg(f + 1);
      ids = l.ids + (int64_t)row * l.K;
      q = l.q + (int64_t)row * l.K;
    }
    load();
  }
  __device__ __forceinline__ void next() {
    ++at;
    load();
  }
};

// ---------------------------------------------------------------- forward
// 8 floats, a whole 32-byte sector in one store: a lane's row is far from the next lane's,
// and with half sectors the forward that keeps its logits took 1.44 ms at N = 2048, H = 4096,
// V = 151936, against 1.25 - 1.37 ms so (1.27 ms without keeping them).
__device__ __forceinline__ void store_sector(float* p, const float* z) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(z[0]),
               "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7])
               : "memory");
}

// sum += x, and what the rounding lost to `lost` (the sum of two numbers is exact in two; NaN
// where an infinity came in).  Hundreds of slots of one vocabulary split, added plainly, were off
// by 4e-5 at logits of 13.
__device__ __forceinline__ void sum_exactly(float x, float& sum, float& lost) {
  const float to = __fadd_rn(sum, x), of_x = __fsub_rn(to, sum);
  lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(sum, __fsub_rn(to, of_x)), __fsub_rn(x, of_x)));
  sum = to;
}

struct DistillArgs {
  int N, V;
  float scale;                // log2(e) / T
  const float* bias;
  bool bias_vec4;
  Lists lists;                // one span per vocabulary split
  float2* ws_ms;              // [N][S]: (m, s)
  float* ws_d;                // [N][S]: sum of q z over the split's slots
  int S;
  float* logits;              // [N][ld_logits] z in FP32, or null; rows of whole sectors
  int64_t ld_logits;
};

// Epilogue warps (2..5) of both loops; the (m, s) arithmetic is the fused linear-logp's.
template <bool kSolo>
__device__ __forceinline__ void distill_epilogue(const VocabSched& sc, const DistillArgs& a,
                                                 const PipeSmem& ps, uint32_t tmem) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int q = warp & 3;
  const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
  int acc = 0;
  uint32_t acc_phase = 0;
  bool run = true;
  for (int k = 0; run; ++k) {
    const int u = kSolo ? solo_unit(sc, k) : warp_unit_take(sc, ps, k, &g_err_linear_distill);
    if (u < 0) break;
    const int j = sc.split_of(u);
    const int row = sc.rb_of(u) * sc.rows_per_unit + (kSolo ? 0 : (int)ps.rank * kHalfRows) +
                    q * 32 + lane;
    const bool valid = row < a.N;
    SlotWalk slot;
    slot.start(a.lists, row, j, valid);
    float m = -INFINITY, s = 0.f, d = 0.f, d_lost = 0.f;
    const int t0 = sc.first_tile(u), nt = sc.unit_tiles(u);
    const bool has_bias = a.bias != nullptr;
    for (int i = 0; i < nt; ++i) {
      const int v0 = (t0 + i) * kBN;
      BiasTile bias;
      if (has_bias) load_bias_tile(a.bias + v0, a.V - v0, a.bias_vec4, lane, bias);
      if (!epilogue_acquire(ps, acc, acc_phase, &g_err_linear_distill)) {
        run = false;
        break;
      }
      const uint32_t taddr = tmem + acc * kAccCols + lane_off;
#pragma unroll 1
      for (int c = 0; c < kBN / 32; ++c) {
        const int vbase = v0 + c * 32;
        if (vbase >= a.V) break;          // uniform: depends on the tile only
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(taddr + c * 32, r);
        tmem_wait_ld();
        float z[32];
        chunk_logits(r, vbase, a.V, has_bias, bias, c, z);
        if (a.logits && valid) {
          float* dst = a.logits + (int64_t)row * a.ld_logits + vbase;
#pragma unroll
          for (int g = 0; g < 4; ++g)   // groups past V stay within ld_logits
            if (vbase + 8 * g < a.V &&
                RLK_STORE_OK(vbase + 8 * g + 8 <= a.ld_logits, &g_err_linear_distill))
              store_sector(dst + 8 * g, z + 8 * g);
        }
        while (__any_sync(0xffffffffu, slot.id < vbase + 32)) {
          if (slot.id < vbase + 32) {
            const float zk = chunk_at(z, slot.id - vbase);
            if (slot.w != 0.f) sum_exactly(__fmul_rn(slot.w, zk), d, d_lost);   // 0 of a banned id is 0
            slot.next();
          }
        }
        chunk_fold(z, a.scale, m, s);
      }
      if (kSolo)
        solo_release(ps, acc);
      else
        epilogue_release(ps, acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (!run) break;
    if (valid && RLK_STORE_OK(row >= 0 && j >= 0 && j < a.S, &g_err_linear_distill)) {
      a.ws_ms[(int64_t)row * a.S + j] = make_float2(m, s);
      a.ws_d[(int64_t)row * a.S + j] = d_lost == d_lost ? __fadd_rn(d, d_lost) : d;
    }
  }
}

// Bound by the tensor cores: the epilogue of one accumulator hides behind the MMAs of the
// other.  2 N H V operations at N = 4096, H = 4096, V = 151936 in 2.75 - 2.9 ms (with the lists and
// the merge; the power cap decides): 1.76 - 1.85 PFLOP/s, 0.94 - 0.99 of a measured library
// product's burst rate; at N = 1024, H = 2048, V = 32003 88 us, 1.52 PFLOP/s.  The split of V and
// the 64 or 128 columns a stage are the fused linear-logp's rules, so lse at T = 1 has its bits.
template <int kK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    distill_partials_kernel(const __grid_constant__ CUtensorMap tm_hidden,
                            const __grid_constant__ CUtensorMap tm_weight, VocabSched sc,
                            DistillArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_hidden);
    tma_prefetch_desc(&tm_weight);
  }
  const uint32_t tmem = pipe_setup(ps);
  using THalf = OperandTile<false, kHalfRows, kK>;
  using R = PairRingT<kHalfRows, kK>;
  if (warp == 0) {
    if (lane == 0)
      producer_role<THalf, THalf, VocabSched, R>(&tm_hidden, &tm_weight, sc, ps,
                                                 &g_err_linear_distill);
    if (lane == 1 && ps.rank == 0) scheduler_role(sc, ps, &g_err_linear_distill);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && ps.rank == 0)
      mma_role<THalf, THalf, VocabSched, R>(sc, ps, tmem,
                                            idesc_bf16_f32(kPairRows, kBN, false, false),
                                            &g_err_linear_distill);
    __syncwarp();
  } else {
    distill_epilogue<false>(sc, args, ps, tmem);
  }
  pipe_teardown(tmem);
}

// At most 128 rows: bound by reading W once.  N = 17, H = 4096, V = 151936 in 180 us, 6.9 TB/s
// (the measured copy: 6.8 TB/s).
template <class R>
__global__ void __launch_bounds__(kThreads, 1)
    distill_solo_kernel(const __grid_constant__ CUtensorMap tm_hidden,
                        const __grid_constant__ CUtensorMap tm_weight, VocabSched sc,
                        DistillArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_hidden);
    tma_prefetch_desc(&tm_weight);
  }
  const uint32_t tmem = solo_setup(ps);
  using TA = OperandTile<false, R::kARows>;
  using TB = OperandTile<false, kBN>;
  if (warp == 0) {
    if (lane == 0) solo_producer<TA, TB, R>(&tm_hidden, &tm_weight, sc, ps, &g_err_linear_distill);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0)
      solo_mma<TA, TB, R>(sc, ps, tmem, idesc_bf16_f32(kHalfRows, kBN, false, false),
                          &g_err_linear_distill);
    __syncwarp();
  } else {
    distill_epilogue<true>(sc, args, ps, tmem);
  }
  solo_teardown(tmem);
}

struct CombineArgs {
  const float2* ms;
  const float* d;
  Lists lists;
  const float* teacher_lse;
  int N, S;
  float temperature, scale;
  double inv_t;
  float* loss;
  float* lse;
};

// One warp per row: (m, s) and D over the splits, lane l taking splits l, l + 32, ...
// ascending, then a xor butterfly of symmetric sums (all lanes end with the same bits); Q over
// the slots alike.  Then a thread per row: with y = (t - top) / T and L the teacher's norm,
//   loss = T^2 (sum q y - (D - M Q) / T + Q (log s - L)),  L = log sum exp y, or lse - top / T.
// T^2 multiplies what the parts lost, and parts of size log V lose 5e-7 each (in FP32, joined
// from lse, the loss was off by 1e-4 at T = 10 and 1e-2 at T = 100 where it is 0.5): so the two
// sums of exponentials meet in one logarithm of their ratio, and the parts are joined in FP64.
// What is left is the error of s, some 2e-7 of T^2.  At T = 1 the rounded lse stands in for
// M + log s, so that one slot gives -logp exactly.
// 12 bytes a split and row; latency: 11 us for 4096 rows of 594 splits (29 MB, from L2).
__global__ void __launch_bounds__(256)
    distill_combine_kernel(const __grid_constant__ CombineArgs a) {
  __shared__ float4 parts[8];                      // M, s, D, Q of the block's rows
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  int row = blockIdx.x * 8 + threadIdx.x;
  const bool ends = threadIdx.x < 8 && row < a.N;  // the row that this thread ends: loads go ahead
  float2 t = make_float2(0.f, 0.f);
  float teacher = 0.f;
  if (ends) {
    t = a.lists.sums[row];
    if (a.teacher_lse) teacher = a.teacher_lse[row];
  }
  row = blockIdx.x * 8 + threadIdx.x / 32;
  if (row < a.N) {
    float M = -INFINITY, s = 0.f, d = 0.f, Q = 0.f;
    const float* q = a.lists.q + (int64_t)row * a.lists.K;
    const float2* ms = a.ms + (int64_t)row * a.S;
    const float* dz = a.d + (int64_t)row * a.S;
#pragma unroll 4
    for (int k = lane; k < a.lists.K; k += 32) Q = __fadd_rn(Q, __ldg(q + k));
    for (int j0 = lane; j0 < a.S; j0 += 128) {     // four splits' loads before the first merge
      float2 v[4];
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = min(j0 + 32 * i, a.S - 1);
        v[i] = __ldg(ms + j);
        x[i] = __ldg(dz + j);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + 32 * i < a.S) {
          merge_ms(M, s, v[i].x, v[i].y, a.scale);
          d = __fadd_rn(d, x[i]);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, off);
      const float s2 = __shfl_xor_sync(0xffffffffu, s, off);
      merge_ms(M, s, m2, s2, a.scale);
      d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, off));
      Q = __fadd_rn(Q, __shfl_xor_sync(0xffffffffu, Q, off));
    }
    if (lane == 0) parts[threadIdx.x / 32] = make_float4(M, s, d, Q);
  }
  __syncthreads();
  row = blockIdx.x * 8 + threadIdx.x;
  if (!ends || !RLK_STORE_OK(row >= 0, &g_err_linear_distill)) return;
  const float4 r = parts[threadIdx.x];
  const float M = r.x, s = r.y, Q = r.w, T = a.temperature;
  const float lse = __fadd_rn(__fdiv_rn(M, T), logf(s));
  float loss = 0.f;                                // no used slot, or none with any weight
  if (Q != 0.f) {
    const double d = r.z - (double)M * Q;
    double ratio;                                  // log s - L
    if (a.teacher_lse) {
      const double norm = teacher - t.y * a.inv_t;
      const float near = (float)norm;
      ratio = T == 1.f ? (double)lse - M - norm
                       : logf(__fmul_rn(s, expf(-near))) - (norm - near);
    } else {
      ratio = T == 1.f ? (double)lse - M - logf(t.y) : logf(__fdiv_rn(s, t.y));
    }
    loss = (float)((double)T * T * (t.x - d * a.inv_t + Q * ratio));
  }
  a.lse[row] = lse;
  a.loss[row] = loss;
}

// ---------------------------------------------------------------- backward
struct DistillGradSched {
  Banded order;    // rows = 256-row blocks (one per CTA pair), cols = 256-id vocabulary tiles
  int* counter;
  int nkb, nkb64;
  __device__ __forceinline__ int num_units() const { return order.count(); }
  __device__ __forceinline__ int unit_tiles(int) const { return 1; }
  __device__ __forceinline__ void tile_coords(int u, int, int& a0, int& b0) const {
    int rb, vt;
    order.unit(u, rb, vt);
    a0 = rb * kPairRows;
    b0 = vt * kBN;
  }
};

struct DistillGradArgs {
  int N, V;
  float temperature, scale;
  const float* bias;
  bool bias_vec4;
  const float* lse;
  const float* grad;
  Lists lists;          // one span per 256-id tile
  uint16_t* G;          // [N, ldG] BF16
  int64_t ldG;          // multiple of 8 elements
  float* sums;          // [ceil(N / 32), ldG] column sums of G over 32 rows, or null
};

// Column sums of a 32 x 32 block held a row per lane: halving exchanges leave lane l
// with column l's sum, added in the same tree order for every column.
__device__ __forceinline__ float column_sums(float (&x)[32], int lane) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = up ? x[i] : x[i + w];
      const float keep = up ? x[i + w] : x[i];
      x[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  return x[0];
}

// The forward's product again, so bound by the tensor cores: N = 2048, H = 4096, V = 151936 in
// 1.34 ms, 1.91 PFLOP/s at the clocks of a launch by itself.  Only when the logits were not
// kept: distill_grad_logits_kernel takes 0.26 ms there (0.35 ms with the column sums).
template <int kK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    distill_grad_kernel(const __grid_constant__ CUtensorMap tm_hidden,
                        const __grid_constant__ CUtensorMap tm_weight, DistillGradSched sc,
                        DistillGradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const PipeSmem ps = pipe_smem(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_hidden);
    tma_prefetch_desc(&tm_weight);
  }
  const uint32_t tmem = pipe_setup(ps);
  using THalf = OperandTile<false, kHalfRows, kK>;
  using R = PairRingT<kHalfRows, kK>;
  if (warp == 0) {
    if (lane == 0)
      producer_role<THalf, THalf, DistillGradSched, R>(&tm_hidden, &tm_weight, sc, ps,
                                                       &g_err_linear_distill);
    if (lane == 1 && ps.rank == 0) scheduler_role(sc, ps, &g_err_linear_distill);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && ps.rank == 0)
      mma_role<THalf, THalf, DistillGradSched, R>(sc, ps, tmem,
                                                  idesc_bf16_f32(kPairRows, kBN, false, false),
                                                  &g_err_linear_distill);
    __syncwarp();
  } else {
    const int q = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int k = 0;; ++k) {
      const int u = warp_unit_take(sc, ps, k, &g_err_linear_distill);
      if (u < 0) break;
      int r0, v0;
      sc.tile_coords(u, 0, r0, v0);
      const int row0 = r0 + (int)ps.rank * kHalfRows + q * 32;
      const int row = row0 + lane;
      const bool valid = row < a.N;
      // read before the accumulator is waited for, so the latency hides behind the MMAs
      SlotWalk slot;
      slot.start(a.lists, row, v0 / kBN, valid);
      float up = 0.f, Q = 0.f, L = 0.f;
      if (valid) {
        up = __fmul_rn(__ldg(a.grad + row), a.temperature);
        Q = __ldg(&a.lists.sums[row].y);
        L = __fmul_rn(__ldg(a.lse + row), a.temperature);
      }
      const bool has_bias = a.bias != nullptr;
      BiasTile bias;
      if (has_bias) load_bias_tile(a.bias + v0, a.V - v0, a.bias_vec4, lane, bias);
      if (!epilogue_acquire(ps, acc, acc_phase, &g_err_linear_distill)) break;
      const bool live = valid && Q != 0.f;
      const uint32_t taddr = tmem + acc * kAccCols + lane_off;
#pragma unroll 1
      for (int c = 0; c < kBN / 32; ++c) {
        const int vbase = v0 + c * 32;
        if (vbase >= a.V) break;                 // uniform: depends on the tile only
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(taddr + c * 32, r);
        tmem_wait_ld();
        float G[32];
        chunk_logits(r, vbase, a.V, has_bias, bias, c, G);
#pragma unroll
        for (int i = 0; i < 32; ++i)             // columns past V: z = -inf, p = 0
          G[i] = __fmul_rn(Q, ex2_approx(__fmul_rn(__fsub_rn(G[i], L), a.scale)));
        while (__any_sync(0xffffffffu, slot.id < vbase + 32)) {
          if (slot.id < vbase + 32) {
            const int di = slot.id - vbase;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i == di) G[i] = __fsub_rn(G[i], slot.w);
            slot.next();
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          G[i] = (live && vbase + i < a.V) ? __fmul_rn(up, G[i]) : 0.f;
        if (valid) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            __nv_bfloat162 b = __floats2bfloat162_rn(G[2 * i], G[2 * i + 1]);
            pk[i] = *reinterpret_cast<uint32_t*>(&b);
          }
          uint4* dst = reinterpret_cast<uint4*>(a.G + (int64_t)row * a.ldG + vbase);
#pragma unroll
          for (int g = 0; g < 4; ++g)   // 8 columns per store; groups past V stay within ldG
            if (vbase + 8 * g < a.V &&
                RLK_STORE_OK(row >= 0 && row < a.N && vbase + 8 * g + 8 <= a.ldG,
                             &g_err_linear_distill))
              dst[g] = make_uint4(pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
        }
        if (a.sums && row0 < a.N) {              // uniform in the warp
          const float s = column_sums(G, lane);
          if (vbase + lane < a.V &&
              RLK_STORE_OK(row0 >= 0 && vbase + lane < a.ldG, &g_err_linear_distill))
            a.sums[(int64_t)(row0 / 32) * a.ldG + vbase + lane] = s;
        }
      }
      epilogue_release(ps, acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  pipe_teardown(tmem);
}

// G from kept logits: a block takes 32 rows of a 256-id tile, a warp a row at a time, 8
// columns a lane.  Each element's operations, and the tree of the 32-row column sums, are
// those of distill_grad_kernel.  Bound by its 4 + 2 bytes an element: 262 us at N = 2048,
// V = 151936, 7.1 TB/s (reads outweigh writes; the measured copy, half and half: 6.8 TB/s);
// 349 us with the column sums, which go through shared memory.
template <bool kSums>
__global__ void __launch_bounds__(256)
    distill_grad_logits_kernel(const float* __restrict__ logits, int64_t ld_logits, int vtiles,
                               DistillGradArgs a) {
  __shared__ float sums[kSums ? 32 : 1][kBN];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int group = blockIdx.x / vtiles, tile = blockIdx.x - group * vtiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = tile * kBN + 8 * lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int in_group = warp + 8 * k, row = group * 32 + in_group;
    float G[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) G[i] = 0.f;
    if (row < a.N && v < a.V) {
      const float* z = logits + (int64_t)row * ld_logits + v;
      const float4 x = __ldcs(reinterpret_cast<const float4*>(z));
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v + 4 < a.V) y = __ldcs(reinterpret_cast<const float4*>(z) + 1);
      const float up = __fmul_rn(__ldg(a.grad + row), a.temperature);
      const float Q = __ldg(&a.lists.sums[row].y);
      const float L = __fmul_rn(__ldg(a.lse + row), a.temperature);
      const float zz[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      if (Q != 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          G[i] = __fmul_rn(Q, ex2_approx(__fmul_rn(__fsub_rn(zz[i], L), a.scale)));
        const uint16_t* f = a.lists.first + (int64_t)row * (a.lists.spans + 1) + tile;
        for (int at = __ldg(f), end = __ldg(f + 1); at < end; ++at) {
          const int di = __ldg(a.lists.ids + (int64_t)row * a.lists.K + at) - v;
          const float w = __ldg(a.lists.q + (int64_t)row * a.lists.K + at);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i == di) G[i] = __fsub_rn(G[i], w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) G[i] = v + i < a.V ? __fmul_rn(up, G[i]) : 0.f;
      }
      uint32_t pk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(G[2 * i], G[2 * i + 1]);
        pk[i] = *reinterpret_cast<uint32_t*>(&b);
      }
      if (RLK_STORE_OK(v + 8 <= a.ldG, &g_err_linear_distill))
        *reinterpret_cast<uint4*>(a.G + (int64_t)row * a.ldG + v) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    if (kSums) {
      float4* to = reinterpret_cast<float4*>(&sums[in_group][8 * lane]);
      to[0] = make_float4(G[0], G[1], G[2], G[3]);
      to[1] = make_float4(G[4], G[5], G[6], G[7]);
    }
  }
  if (kSums) {
    __syncthreads();
    float t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) t[r] = __fadd_rn(sums[r][threadIdx.x], sums[r + 16][threadIdx.x]);
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
      for (int r = 0; r < w; ++r) t[r] = __fadd_rn(t[r], t[r + w]);
    const int col = tile * kBN + threadIdx.x;
    if (col < a.V && RLK_STORE_OK(col < a.ldG, &g_err_linear_distill))
      a.sums[(int64_t)group * a.ldG + col] = t[0];
  }
}

// grad_bias[v] = the 32-row sums of column v, in ascending order: 4 N V / 32 bytes, 10 us at
// N = 2048, V = 151936 (3.9 TB/s).
__global__ void __launch_bounds__(256)
    distill_bias_kernel(const float* __restrict__ sums, int groups, int V, int64_t ld,
                        float* __restrict__ out) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int v = blockIdx.x * blockDim.x + threadIdx.x;
  if (v >= V) return;
  float s = 0.f;
#pragma unroll 8
  for (int g = 0; g < groups; ++g) s = __fadd_rn(s, __ldg(sums + g * ld + v));
  if (RLK_STORE_OK(v < V, &g_err_linear_distill)) out[v] = s;
}

// ---------------------------------------------------------------- host side
std::mutex g_attr_mutex;
bool g_attr_set[64];

template <class F>
cudaError_t allow_smem(F* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t ensure_attrs(int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_attr_set[dev]) return cudaSuccess;
  using R64 = PairRingT<kHalfRows, 64>;
  using R128 = PairRingT<kHalfRows, 128>;
  cudaError_t e;
  if ((e = allow_smem(distill_partials_kernel<64>, R64::kSmemBytes)) != cudaSuccess ||
      (e = allow_smem(distill_partials_kernel<128>, R128::kSmemBytes)) != cudaSuccess ||
      (e = allow_smem(distill_solo_kernel<SoloFull>, SoloFull::kSmemBytes)) != cudaSuccess ||
      (e = allow_smem(distill_solo_kernel<SoloThin>, SoloThin::kSmemBytes)) != cudaSuccess ||
      (e = allow_smem(distill_grad_kernel<64>, R64::kSmemBytes)) != cudaSuccess ||
      (e = allow_smem(distill_grad_kernel<128>, R128::kSmemBytes)) != cudaSuccess)
    return e;
  g_attr_set[dev] = true;
  return cudaSuccess;
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Workspace, forward: [ms][D][unit counter][lists][staged hidden][staged W]; backward:
// [G][32-row sums][unit counter][lists][staged hidden][staged W].  Each region starts
// on a 256-byte boundary.
struct DistillPlan {
  int64_t S = 0, vps = 0, vtiles = 0, spans = 0, ldG = 0;
  bool stage_h = false, stage_w = false;
  int64_t ldh = 0, ldw = 0;
  size_t off_a = 0, off_ctr = 0, off_ids = 0, off_q = 0, off_first = 0, off_sums = 0, off_h = 0,
         off_w = 0, total = 0;
};

rlk_status distill_plan(const void* hidden, int64_t N, int64_t H, int64_t ld_hidden,
                        const void* weight, int64_t V, int64_t ld_weight, int64_t K, bool backward,
                        bool want_bias, DistillPlan* p) {
  if (N < 0 || N >= kMaxExtent || H < 1 || H >= (int64_t(1) << 20) || V < 1 ||
      V >= kMaxExtent || ld_hidden < H || ld_weight < H || ld_hidden >= kLdLimit ||
      ld_weight >= kLdLimit || K < 0 || K > kMaxSlots)
    return RLK_ERR_SHAPE;
  rlk_status st = rlk_vocab_split_policy(V, &p->S, &p->vps, &p->vtiles);
  if (st != RLK_OK) return st;
  // work units are numbered in ints (the products: their narrower, 128-column tiles)
  const int64_t rb = ceil_div(N, kPairRows), hb = ceil_div(H, kBN / 2);
  if (rb * p->S >= kUnitLimit) return RLK_ERR_SHAPE;
  if (backward && (ceil_div(N, 32) * p->vtiles >= kUnitLimit || rb * hb >= kUnitLimit ||
                   p->vtiles * hb >= kUnitLimit))
    return RLK_ERR_SHAPE;
  p->spans = backward ? p->vtiles : p->S;
  p->ldG = ceil_div(V, 8) * 8;
  p->stage_h = N > 0 && !tma_ready(hidden, ld_hidden);
  p->stage_w = N > 0 && !tma_ready(weight, ld_weight);
  p->ldh = p->stage_h ? staged_ld(H) : ld_hidden;
  p->ldw = p->stage_w ? staged_ld(H) : ld_weight;
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  if (backward) {
    take((size_t)N * p->ldG * 2);
    p->off_a = take(want_bias ? (size_t)ceil_div(N, 32) * p->ldG * sizeof(float) : 0);
  } else {
    take((size_t)N * p->S * sizeof(float2));
    p->off_a = take((size_t)N * p->S * sizeof(float));
  }
  p->off_ctr = take(256);
  p->off_ids = take((size_t)N * K * sizeof(int));
  p->off_q = take((size_t)N * K * sizeof(float));
  p->off_first = take((size_t)N * (p->spans + 1) * sizeof(uint16_t));
  p->off_sums = take((size_t)N * sizeof(float2));
  p->off_h = take(p->stage_h ? (size_t)N * p->ldh * 2 : 0);
  p->off_w = take(p->stage_w ? (size_t)V * p->ldw * 2 : 0);
  p->total = off;
  return RLK_OK;
}

struct Teacher {
  const int64_t* ids;
  int64_t ld_ids;
  const void* logits;
  int dtype;
  int64_t ld_logits, K;
  const float* lse;
  float temperature;
};

// Sizes and scalars first, then (for calls with rows) pointers.
rlk_status check_teacher(const Teacher& t, int64_t N, bool pointers) {
  if (!pointers) {
    if (t.K < 0 || t.K > kMaxSlots || t.ld_ids < t.K || t.ld_logits < t.K ||
        t.ld_ids >= kLdLimit || t.ld_logits >= kLdLimit)
      return RLK_ERR_SHAPE;
    if (t.dtype != RLK_BF16 && t.dtype != RLK_FP32) return RLK_ERR_DTYPE;
    if (!(t.temperature >= 1e-4f && t.temperature <= 100.f)) return RLK_ERR_VALUE;
    return RLK_OK;
  }
  if (N > 0 && t.K > 0 && (!t.ids || !t.logits)) return RLK_ERR_NULL;
  if (!aligned_to(t.ids, 8) || !aligned_to(t.logits, t.dtype == RLK_FP32 ? 4 : 2) ||
      !aligned_to(t.lse, 4))
    return RLK_ERR_ALIGN;
  return RLK_OK;
}

// Kept logits: rows of whole 32-byte sectors.
rlk_status check_logits(const float* logits, int64_t ld, int64_t V) {
  if (!logits) return RLK_OK;
  if (ld < V || ld % 8 != 0 || ld >= kLdLimit) return RLK_ERR_SHAPE;
  return aligned_to(logits, 32) ? RLK_OK : RLK_ERR_ALIGN;
}

Lists lists_at(uint8_t* ws, const DistillPlan& p, int64_t K, int64_t span) {
  Lists l;
  l.ids = reinterpret_cast<int*>(ws + p.off_ids);
  l.q = reinterpret_cast<float*>(ws + p.off_q);
  l.first = reinterpret_cast<uint16_t*>(ws + p.off_first);
  l.sums = reinterpret_cast<float2*>(ws + p.off_sums);
  l.K = (int)K;
  l.spans = (int)p.spans;
  l.span = span;
  return l;
}

cudaError_t launch_lists(const Teacher& t, int64_t N, int64_t V, const Lists& l, bool backward,
                         cudaStream_t s) {
  ListArgs a;
  a.ids = t.ids;
  a.ld_ids = t.ld_ids;
  a.logits = t.logits;
  a.ld_logits = t.ld_logits;
  a.logits_fp32 = t.dtype == RLK_FP32;
  a.lse = t.lse;
  a.temperature = t.temperature;
  a.inv_t = 1.0 / t.temperature;
  a.N = (int)N;
  a.V = (int)V;
  a.backward = backward;
  const int threads = t.K <= 64 ? 64 : (t.K <= 128 ? 128 : 256);
  return launch_overlapped(distill_lists_kernel, dim3((unsigned)N), threads, 12 * (size_t)t.K, s, a,
                           l);
}

rlk_status cuda_failed() {
  cudaGetLastError();
  return RLK_ERR_CUDA;
}

// Padded copies of what TMA cannot read in place, and the addresses to read from.
rlk_status stage_operands(const void* hidden, int64_t N, int64_t H, int64_t ld_hidden,
                          const void* weight, int64_t V, int64_t ld_weight, const DistillPlan& p,
                          uint8_t* ws, cudaStream_t s, const void** h, const void** w) {
  *h = hidden;
  *w = weight;
  if (p.stage_h) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + p.off_h);
    if (launch_stage_bf16(static_cast<const uint16_t*>(hidden), N, H, ld_hidden, to, p.ldh, s) !=
        cudaSuccess)
      return cuda_failed();
    *h = to;
  }
  if (p.stage_w) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + p.off_w);
    if (launch_stage_bf16(static_cast<const uint16_t*>(weight), V, H, ld_weight, to, p.ldw, s) !=
        cudaSuccess)
      return cuda_failed();
    *w = to;
  }
  return RLK_OK;
}

rlk_status distill_forward(const void* hidden, int64_t N, int64_t H, int64_t ld_hidden,
                           const void* weight, int64_t V, int64_t ld_weight, const float* bias,
                           const Teacher& t, float* loss, float* lse, float* logits,
                           int64_t ld_out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  DistillPlan p;
  rlk_status st =
      distill_plan(hidden, N, H, ld_hidden, weight, V, ld_weight, t.K, false, false, &p);
  if (st != RLK_OK) return st;
  if ((st = check_teacher(t, N, false)) != RLK_OK) return st;
  if ((st = check_logits(logits, ld_out, V)) != RLK_OK) return st;
  if (N == 0) return RLK_OK;
  if (!hidden || !weight || !loss || !lse) return RLK_ERR_NULL;
  if ((st = check_teacher(t, N, true)) != RLK_OK) return st;
  if (!aligned_to(hidden, 2) || !aligned_to(weight, 2) || !aligned_to(bias, 4) ||
      !aligned_to(loss, 4) || !aligned_to(lse, 4))
    return RLK_ERR_ALIGN;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.total)
    return RLK_ERR_WORKSPACE;
  DeviceInfo dev;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  if (ensure_attrs(dev.device) != cudaSuccess) return cuda_failed();

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void *h, *w;
  if ((st = stage_operands(hidden, N, H, ld_hidden, weight, V, ld_weight, p, ws, s, &h, &w)) !=
      RLK_OK)
    return st;
  // The loops, rings and stage depths are the fused linear-logp's, for its reasons.
  const bool solo = N <= kHalfRows, thin = N <= 32;
  const int rows_per_unit = solo ? kHalfRows : kPairRows;
  CUtensorMap tm_h, tm_w;
  if (!encode_bf16_2d(&tm_h, h, H, N, p.ldh, kBK, thin ? 32 : kHalfRows) ||
      !encode_bf16_2d(&tm_w, w, H, V, p.ldw, kBK, solo ? kBN : kHalfRows))
    return RLK_ERR_CUDA;
  const Lists lists = lists_at(ws, p, t.K, p.vps * kVocabTile);
  if (launch_lists(t, N, V, lists, false, s) != cudaSuccess) return cuda_failed();

  VocabSched sc;
  sc.order.rows = (int)ceil_div(N, rows_per_unit);
  sc.order.cols = (int)p.S;
  sc.order.band = band_rows(sc.order.rows, H, rows_per_unit);
  sc.rows_per_unit = rows_per_unit;
  sc.S = (int)p.S;
  sc.vps = (int)p.vps;
  sc.vtiles = (int)p.vtiles;
  sc.tile0 = 0;
  const int stage_k = !solo && N > kWideStageRows ? 128 : 64;
  sc.nkb = (int)ceil_div(H, stage_k);
  sc.nkb64 = (int)ceil_div(H, kBK);
  sc.counter = nullptr;
  DistillArgs a;
  a.N = (int)N;
  a.V = (int)V;
  a.scale = kLog2e / t.temperature;
  a.bias = bias;
  a.bias_vec4 = aligned_to(bias, 16);
  a.lists = lists;
  a.ws_ms = reinterpret_cast<float2*>(ws);
  a.ws_d = reinterpret_cast<float*>(ws + p.off_a);
  a.S = (int)p.S;
  a.logits = logits;
  a.ld_logits = ld_out;
  const int64_t units = (int64_t)sc.order.rows * sc.S;
  cudaError_t e;
  if (solo) {
    const int grid = (int)(units < dev.sm_count ? units : dev.sm_count);
    e = thin ? launch_overlapped(distill_solo_kernel<SoloThin>, grid, kThreads,
                                 SoloThin::kSmemBytes, s, tm_h, tm_w, sc, a)
             : launch_overlapped(distill_solo_kernel<SoloFull>, grid, kThreads,
                                 SoloFull::kSmemBytes, s, tm_h, tm_w, sc, a);
  } else {
    const int64_t clusters = dev.sm_count / 2;
    const int grid = 2 * (int)(units < clusters ? units : clusters);
    if (ordered_units(units, clusters)) {
      sc.counter = reinterpret_cast<int*>(ws + p.off_ctr);
      if (cudaMemsetAsync(sc.counter, 0, sizeof(int), s) != cudaSuccess) return cuda_failed();
    }
    e = stage_k == 128
            ? launch_overlapped(distill_partials_kernel<128>, grid, kThreads,
                                PairRingT<kHalfRows, 128>::kSmemBytes, s, tm_h, tm_w, sc, a)
            : launch_overlapped(distill_partials_kernel<64>, grid, kThreads,
                                PairRingT<kHalfRows, 64>::kSmemBytes, s, tm_h, tm_w, sc, a);
  }
  if (e != cudaSuccess) return cuda_failed();
  CombineArgs c;
  c.ms = a.ws_ms;
  c.d = a.ws_d;
  c.lists = lists;
  c.teacher_lse = t.lse;
  c.N = (int)N;
  c.S = (int)p.S;
  c.temperature = t.temperature;
  c.scale = a.scale;
  c.inv_t = 1.0 / t.temperature;
  c.loss = loss;
  c.lse = lse;
  if (launch_overlapped(distill_combine_kernel, (int)ceil_div(N, 8), 256, 0, s, c) != cudaSuccess)
    return cuda_failed();
  return RLK_OK;
}

}  // namespace

uint32_t take_error_linear_distill() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_linear_distill, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaMemcpyToSymbol(g_err_linear_distill, &zero, sizeof zero);
  cudaGetLastError();
  return v;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

size_t rlk_linear_distill_workspace_size(const void* hidden, int64_t N, int64_t H,
                                         int64_t ld_hidden, const void* weight, int64_t V,
                                         int64_t ld_weight, int64_t K) {
  DistillPlan p;
  if (distill_plan(hidden, N, H, ld_hidden, weight, V, ld_weight, K, false, false, &p) != RLK_OK)
    return 0;
  return p.total;
}

rlk_status rlk_linear_distill(const void* hidden, int64_t N, int64_t H, int64_t ld_hidden,
                              const void* weight, int64_t V, int64_t ld_weight, const float* bias,
                              const int64_t* teacher_ids, int64_t ld_ids,
                              const void* teacher_logits, int logits_dtype, int64_t ld_logits,
                              int64_t K, const float* teacher_lse, float temperature, float* loss,
                              float* lse, float* logits, int64_t ld_logits_out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  RLK_CALL_RANGE();
  const Teacher t = {teacher_ids, ld_ids,      teacher_logits, logits_dtype,
                     ld_logits,   K,           teacher_lse,    temperature};
  return distill_forward(hidden, N, H, ld_hidden, weight, V, ld_weight, bias, t, loss, lse, logits,
                         ld_logits_out, workspace, workspace_bytes, stream);
}

size_t rlk_linear_distill_backward_workspace_size(const void* hidden, int64_t N, int64_t H,
                                                  int64_t ld_hidden, const void* weight, int64_t V,
                                                  int64_t ld_weight, int64_t K, int want_bias) {
  DistillPlan p;
  if (distill_plan(hidden, N, H, ld_hidden, weight, V, ld_weight, K, true, want_bias != 0, &p) !=
      RLK_OK)
    return 0;
  return p.total;
}

rlk_status rlk_linear_distill_backward(
    const void* hidden, int64_t N, int64_t H, int64_t ld_hidden, const void* weight, int64_t V,
    int64_t ld_weight, const float* bias, const int64_t* teacher_ids, int64_t ld_ids,
    const void* teacher_logits, int logits_dtype, int64_t ld_logits, int64_t K,
    const float* teacher_lse, float temperature, const float* lse, const float* kept_logits,
    int64_t ld_kept, const float* grad_loss, void* grad_hidden, int grad_hidden_dtype, int64_t ld_grad_hidden, void* grad_weight,
    int grad_weight_dtype, int64_t ld_grad_weight, float* grad_bias, void* workspace,
    size_t workspace_bytes, void* stream) {
  RLK_CALL_RANGE();
  // ---- every check, including those of the products below, before the first launch
  const Teacher t = {teacher_ids, ld_ids,      teacher_logits, logits_dtype,
                     ld_logits,   K,           teacher_lse,    temperature};
  DistillPlan p;
  rlk_status st = distill_plan(hidden, N, H, ld_hidden, weight, V, ld_weight, K, true,
                               grad_bias != nullptr, &p);
  if (st != RLK_OK) return st;
  if ((st = check_teacher(t, N, false)) != RLK_OK) return st;
  if ((st = check_logits(kept_logits, ld_kept, V)) != RLK_OK) return st;
  if (grad_hidden && (ld_grad_hidden < H || ld_grad_hidden >= kLdLimit)) return RLK_ERR_SHAPE;
  if (grad_weight && (ld_grad_weight < H || ld_grad_weight >= kLdLimit)) return RLK_ERR_SHAPE;
  if ((grad_hidden && grad_hidden_dtype != RLK_BF16 && grad_hidden_dtype != RLK_FP32) ||
      (grad_weight && grad_weight_dtype != RLK_BF16 && grad_weight_dtype != RLK_FP32))
    return RLK_ERR_DTYPE;
  const size_t es_h = grad_hidden_dtype == RLK_FP32 ? 4 : 2;
  const size_t es_w = grad_weight_dtype == RLK_FP32 ? 4 : 2;
  if ((grad_hidden && !aligned_to(grad_hidden, es_h)) ||
      (grad_weight && !aligned_to(grad_weight, es_w)) || !aligned_to(grad_bias, 4))
    return RLK_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (N == 0) {
    // No rows: grad_hidden is empty; grad_weight and grad_bias are the empty sums.
    if (!grad_weight && !grad_bias) return RLK_OK;
    if ((st = device_ready(&dev)) != RLK_OK) return st;
    if ((grad_weight && cudaMemset2DAsync(grad_weight, ld_grad_weight * es_w, 0, H * es_w, V, s) !=
                            cudaSuccess) ||
        (grad_bias && cudaMemsetAsync(grad_bias, 0, V * sizeof(float), s) != cudaSuccess))
      return cuda_failed();
    return RLK_OK;
  }
  if (!hidden || !weight || !lse || !grad_loss) return RLK_ERR_NULL;
  if ((st = check_teacher(t, N, true)) != RLK_OK) return st;
  if (!aligned_to(hidden, 2) || !aligned_to(weight, 2) || !aligned_to(lse, 4) ||
      !aligned_to(grad_loss, 4) || !aligned_to(bias, 4))
    return RLK_ERR_ALIGN;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.total)
    return RLK_ERR_WORKSPACE;
  if ((st = device_ready(&dev)) != RLK_OK) return st;
  if (ensure_attrs(dev.device) != cudaSuccess) return cuda_failed();
  if (!grad_hidden && !grad_weight && !grad_bias) return RLK_OK;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void *h, *w;
  if ((st = stage_operands(hidden, N, H, ld_hidden, weight, V, ld_weight, p, ws, s, &h, &w)) !=
      RLK_OK)
    return st;
  CUtensorMap tm_h, tm_w;
  if (!encode_bf16_2d(&tm_h, h, H, N, p.ldh, kBK, kHalfRows) ||
      !encode_bf16_2d(&tm_w, w, H, V, p.ldw, kBK, kHalfRows))
    return RLK_ERR_CUDA;
  const Lists lists = lists_at(ws, p, K, kVocabTile);
  if (launch_lists(t, N, V, lists, true, s) != cudaSuccess) return cuda_failed();

  DistillGradSched sc;
  sc.order.rows = (int)ceil_div(N, kPairRows);
  sc.order.cols = (int)p.vtiles;
  sc.order.band = band_rows(sc.order.rows, H, kPairRows);
  const int stage_k = N > kWideStageRows ? 128 : 64;
  sc.nkb = (int)ceil_div(H, stage_k);
  sc.nkb64 = (int)ceil_div(H, kBK);
  sc.counter = nullptr;
  DistillGradArgs a;
  a.N = (int)N;
  a.V = (int)V;
  a.temperature = temperature;
  a.scale = kLog2e / temperature;
  a.bias = bias;
  a.bias_vec4 = aligned_to(bias, 16);
  a.lse = lse;
  a.grad = grad_loss;
  a.lists = lists;
  a.G = reinterpret_cast<uint16_t*>(ws);
  a.ldG = p.ldG;
  a.sums = grad_bias ? reinterpret_cast<float*>(ws + p.off_a) : nullptr;
  const int64_t units = (int64_t)sc.order.rows * sc.order.cols;
  const int64_t clusters = dev.sm_count / 2;
  const int grid = 2 * (int)(units < clusters ? units : clusters);
  int* counter = reinterpret_cast<int*>(ws + p.off_ctr);
  cudaError_t e;
  if (kept_logits) {
    const dim3 blocks((unsigned)(ceil_div(N, 32) * p.vtiles));
    e = a.sums ? launch_overlapped(distill_grad_logits_kernel<true>, blocks, 256, 0, s, kept_logits,
                                   ld_kept, (int)p.vtiles, a)
               : launch_overlapped(distill_grad_logits_kernel<false>, blocks, 256, 0, s, kept_logits,
                                   ld_kept, (int)p.vtiles, a);
  } else {
    if (ordered_units(units, clusters)) {
      sc.counter = counter;
      if (cudaMemsetAsync(sc.counter, 0, sizeof(int), s) != cudaSuccess) return cuda_failed();
    }
    e = stage_k == 128
            ? launch_overlapped(distill_grad_kernel<128>, grid, kThreads,
                                PairRingT<kHalfRows, 128>::kSmemBytes, s, tm_h, tm_w, sc, a)
            : launch_overlapped(distill_grad_kernel<64>, grid, kThreads,
                                PairRingT<kHalfRows, 64>::kSmemBytes, s, tm_h, tm_w, sc, a);
  }
  if (e != cudaSuccess) return cuda_failed();

  // G and the (possibly staged) operands are TMA-ready and every argument of the
  // products was checked above.  One launch or two: the linear-logp backward's rule.
  const int64_t long_tiles = ceil_div(V >= N ? N : V, kPairRows) * ceil_div(H, kBN);
  if (grad_hidden && grad_weight && 2 * long_tiles <= dev.sm_count / 2) {
    st = launch_fwd_and_db(a.G, N, V, a.ldG, w, H, p.ldw, grad_hidden, grad_hidden_dtype,
                           ld_grad_hidden, h, p.ldh, grad_weight, grad_weight_dtype,
                           ld_grad_weight, counter, s);
    if (st != RLK_OK) return st;
  } else {
    if (grad_hidden) {   // [N, H] = G [N, V] . W [V, H]
      st = rlk_det_gemm_fwd(a.G, N, V, a.ldG, w, H, p.ldw, grad_hidden, grad_hidden_dtype,
                            ld_grad_hidden, nullptr, 0, stream);
      if (st != RLK_OK) return st;
    }
    if (grad_weight) {   // [V, H] = G^T . hidden
      st = rlk_det_gemm_db(a.G, N, V, a.ldG, h, RLK_BF16, H, p.ldh, grad_weight,
                           grad_weight_dtype, ld_grad_weight, nullptr, 0, stream);
      if (st != RLK_OK) return st;
    }
  }
  if (grad_bias && launch_overlapped(distill_bias_kernel, (int)ceil_div(V, 256), 256, 0, s, a.sums,
                                     (int)ceil_div(N, 32), (int)V, a.ldG, grad_bias) != cudaSuccess)
    return cuda_failed();
  return RLK_OK;
}

}  // extern "C"
