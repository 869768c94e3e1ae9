// Sampling one token a row from logits with temperature, top-k, top-p and min-p, from one
// given uniform number a row, on sm_103a.
//
// Row z[0 .. V), top m = max z, temperature T, c = log2(e) / T:
//   x_v = max((z_v - m) c, -126),   w_v = 2^x_v as a multiple of 2^-31 (a whole number)
// In descending order of z, equal logits by id, keep v when
//   top-k   fewer than k come before it,
//   top-p   the weights before it sum to less than P = max(1, floor(p C_k)), C_k = the
//           weight of the k kept by top-k, p a multiple of 2^-24,
//   min-p   w_v >= min_p 2^31.
// With C = the weight kept and t = floor(floor(u 2^31) C / 2^31), the token is the first id
// whose running sum of kept weights, by id, exceeds t; logp = (z - m) / T - log(C / 2^31).
//
// Every operation up to w is one rounded FP32 operation and every sum after it is of whole
// numbers, so the token depends on nothing but the row: any split of the row, any order
// and any cluster size give it.  2^f on [-1/2, 1/2] is a polynomial fitted by least squares
// of the relative error (below 2e-7), its products and sums rounded one by one.  A weight
// below 2^-32 of the largest is 0; u's own steps are 2^-31.
//
// The row is read once from memory (the bound: V elements) and stays on chip: a cluster of
// 1 - 16 CTAs holds it in shared memory, each CTA a contiguous run of ids, and passes over
// it there.  After the maximum, rows with top-k or top-p find where the kept prefix of the
// sorted order ends without sorting the row: a histogram of x over 16 octaves (counts, and
// weights for top-p), whose bins are runs of the sorted order, gives the bin the cut falls
// in.  If what lies up to that bin is at most kList elements, the leading CTA sorts just
// those and finishes; otherwise the cut is narrowed inside the bin by histograms of the
// logits' bit patterns to one value, then one id among equal values.
#include <math.h>

#include <mutex>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_pipeline.cuh"

namespace rlk {

__device__ unsigned int g_err_sample = 0;

namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 1024;                  // histogram bins; two per thread in the scan
constexpr int kList = 2048;                  // candidates the leading CTA sorts
constexpr int kMaxCluster = 16;
constexpr int64_t kMaxSampleVocab = 524288;
constexpr float kWindow = 16.f;              // octaves of x per histogram window
constexpr int kWindows = 2;                  // weights vanish below 2^-32
constexpr uint32_t kOne = 1u << 31;
constexpr uint32_t kFull = 0xffffffffu;

static_assert(kBins == 2 * kSampleThreads, "the scan takes two bins per thread");

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int N, V;
  const float* temperature;   // per row, or null: the one value
  const int* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  const void* uniform;
  int uniform_fp64;
  int64_t* token;
  float* logp;
};

// ---------------------------------------------------------------- weights
__device__ __forceinline__ float x_of(float z, float m, float c) {
  return fmaxf(__fmul_rn(__fsub_rn(z, m), c), -126.f);
}

// 2^(x + 31) rounded to a whole number (nearest even), x in [-126, 0].
__device__ __forceinline__ uint32_t weight_of(float x) {
  constexpr float kRound = 12582912.f;       // 1.5 * 2^23: adding it rounds to a whole number
  const float t = __fadd_rn(x, kRound);
  const float f = __fsub_rn(x, __fsub_rn(t, kRound));
  float y = 0.0013264727313071489f;
  y = __fadd_rn(__fmul_rn(y, f), 0.009671512991189957f);
  y = __fadd_rn(__fmul_rn(y, f), 0.05550733581185341f);
  y = __fadd_rn(__fmul_rn(y, f), 0.24022242426872253f);
  y = __fadd_rn(__fmul_rn(y, f), 0.6931470036506653f);
  y = __fadd_rn(__fmul_rn(y, f), 1.f);
  const int n = __float_as_int(t) - __float_as_int(kRound) + 31;
  return __float2uint_rn(__int_as_float(__float_as_int(y) + (n << 23)));
}

// Order-preserving bit pattern of a logit (+0 and -0 alike).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.f));
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Bin of x in the window [-(w + 1) kWindow, -w kWindow): 0 .. kBins - 1 inside, negative
// above, kBins or more below.  Falls with x, so a bin is a run of the sorted order.
__device__ __forceinline__ int bin_of(float x, int window) {
  return __float2int_rd(__fmul_rn(__fsub_rn(-kWindow * window, x), kBins / kWindow));
}

// floor(a b / 2^31) and floor(a p / 2^24), a < 2^50, b < 2^31, p <= 2^24, exactly.
__device__ __forceinline__ uint64_t scaled_31(uint64_t a, uint32_t b) {
  return (a >> 31) * b + (((a & (kOne - 1)) * b) >> 31);
}
__device__ __forceinline__ uint64_t scaled_24(uint64_t a, uint32_t p) {
  return (((a >> 31) * p) << 7) + (((a & (kOne - 1)) * p) >> 24);
}

// ---------------------------------------------------------------- the row on chip
// The row in 16-byte vectors of its memory: element j of the vectors is id j - lead, where
// lead (< one vector) is how far the row's start lies past a 16-byte boundary; elements
// outside the row are -inf.  The CTA of rank r holds vectors [r * per, (r + 1) * per); in
// every pass, warp w takes a contiguous part of them, a vector per lane and step, so the
// order (CTA, warp, step, lane, element) is the order of ids.
template <bool kFp32>
struct Row {
  static constexpr int kElems = kFp32 ? 4 : 8;
  const uint4* smem;     // this CTA's vectors
  int first_id;          // id of the CTA's element 0
  int v0, v1;            // this warp's vectors

  __device__ __forceinline__ void get(int v, float (&z)[kElems]) const { unpack(smem[v], z); }
  static __device__ __forceinline__ void unpack(const uint4& q, float (&z)[kElems]) {
    const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kFp32) {
        z[i] = __uint_as_float(r[i]);
      } else {
        z[2 * i] = __uint_as_float(r[i] << 16);
        z[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  }
};

// ---------------------------------------------------------------- cluster exchange
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t atom_add_cluster(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(addr), "r"(v)
               : "memory");
  return old;
}

// Cluster barrier after code in which a warp's lanes may have parted.
__device__ __forceinline__ void cluster_join() {
  __syncwarp();
  cluster_sync();
}

struct Cut {             // where a search ended
  int bin;               // -1: not in this histogram
  uint32_t before, in;   // elements in the bins before it, and in it
  uint64_t mass;         // weight of the bins before it
};

// Fixed shared memory; the row's vectors follow.  The candidates take the histogram's
// place: they are pushed after the second barrier of find_cut, past which no CTA reads
// another's histogram.
struct SampleSmem {
  union {
    struct {
      uint32_t count[kBins], lo[kBins], hi[kBins];   // this CTA's; weights as two halves
    };
    uint64_t list[kList];                        // candidates (in the leading CTA)
  };
  uint64_t slice_mass[kBins];                    // merged: this CTA's 1 / C of the bins
  uint32_t slice_count[kBins];
  uint64_t part[8][kSampleWarps];                // block reductions
  uint64_t xch[8];                               // a CTA's values for its peers, a slot a step
  uint64_t xmass[4];
  Cut cut;
  uint32_t n_list;
  int answer;
};

struct Block {
  SampleSmem* s;
  int rank, ctas;
  __device__ __forceinline__ uint32_t peer(const void* p, int r) const {
    return mapa_shared(smem_u32(p), (uint32_t)r);
  }
};

// Sum of v over the block; every thread gets it.  `slot`: one of the part rows, not used
// again before the next __syncthreads.
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

__device__ __forceinline__ uint64_t block_sum(const Block& b, uint64_t v, int slot) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) b.s->part[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kSampleWarps; ++w) v += b.s->part[slot][w];
  return v;
}

// Inclusive prefix sums over the block's threads of (count, mass).
__device__ __forceinline__ void block_scan(const Block& b, uint32_t& n, uint64_t& m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t n2 = __shfl_up_sync(kFull, n, off);
    const uint64_t m2 = __shfl_up_sync(kFull, m, off);
    if (lane >= off) {
      n += n2;
      m += m2;
    }
  }
  __syncthreads();
  if (lane == 31) {
    b.s->part[6][warp] = n;
    b.s->part[7][warp] = m;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    n += (uint32_t)b.s->part[6][w];
    m += b.s->part[7][w];
  }
}

__device__ __forceinline__ void clear_bins(const Block& b, bool mass) {
  for (int i = threadIdx.x; i < kBins; i += kSampleThreads) {
    b.s->count[i] = 0;
    if (mass) {
      b.s->lo[i] = 0;
      b.s->hi[i] = 0;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void add_to_bin(const Block& b, int bin, bool mass, uint32_t w) {
  atomicAdd(&b.s->count[bin], 1u);
  if (mass) {
    atomicAdd(&b.s->lo[bin], w & 0xffffu);      // a CTA holds at most 2^15 elements
    atomicAdd(&b.s->hi[bin], w >> 16);
  }
}

// The first bin at which the running count reaches want_count, or (by_mass) the running
// weight reaches want_mass, over the cluster's histograms; *all receives the totals.
__device__ __forceinline__ Cut find_cut(const Block& b, bool mass, bool by_mass,
                                        uint32_t want_count, uint64_t want_mass, uint32_t* all_n,
                                        uint64_t* all_mass) {
  SampleSmem* s = b.s;
  const int per = kBins / b.ctas;
  cluster_join();                                // every CTA's histogram is complete
  for (int i = threadIdx.x; i < per; i += kSampleThreads) {
    const int bin = b.rank * per + i;
    uint32_t n = 0;
    uint64_t m = 0;
    for (int r = 0; r < b.ctas; ++r) {
      n += ld_cluster_u32(b.peer(&s->count[bin], r));
      if (mass)
        m += ld_cluster_u32(b.peer(&s->lo[bin], r)) +
             ((uint64_t)ld_cluster_u32(b.peer(&s->hi[bin], r)) << 16);
    }
    s->slice_count[i] = n;
    s->slice_mass[i] = m;
  }
  if (threadIdx.x == 0) s->cut.bin = -1;
  cluster_join();                                // every slice is merged
  const int bin = 2 * threadIdx.x;
  const int owner = bin / per, at = bin - owner * per;   // per is even: both bins have one owner
  uint32_t n[2];
  uint64_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    n[i] = ld_cluster_u32(b.peer(&s->slice_count[at + i], owner));
    m[i] = mass ? ld_cluster_u64(b.peer(&s->slice_mass[at + i], owner)) : 0;
  }
  uint32_t cn = n[0] + n[1];
  uint64_t cm = m[0] + m[1];
  block_scan(b, cn, cm);                         // inclusive, through this thread's two bins
  uint32_t bn = cn - n[0] - n[1];
  uint64_t bm = cm - m[0] - m[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool was = by_mass ? bm >= want_mass : bn >= want_count;
    const bool is = by_mass ? bm + m[i] >= want_mass : bn + n[i] >= want_count;
    if (!was && is) s->cut = Cut{bin + i, bn, n[i], bm};
    bn += n[i];
    bm += m[i];
  }
  if (threadIdx.x == kSampleThreads - 1) {
    s->part[4][0] = cn;
    s->part[4][1] = cm;
  }
  __syncthreads();
  *all_n = (uint32_t)s->part[4][0];
  *all_mass = s->part[4][1];
  return s->cut;
}

// Ascending bitonic sort of n (a power of two) 64-bit values in shared memory.
__device__ __forceinline__ void block_sort(uint64_t* a, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int step = size >> 1; step >= 1; step >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += kSampleThreads) {
        const int i = 2 * t - (t & (step - 1)), j = i + step;
        const uint64_t x = a[i], y = a[j];
        if ((x > y) == ((i & size) == 0)) {
          a[i] = y;
          a[j] = x;
        }
      }
      __syncthreads();
    }
}

struct Filter {
  float m, c, tau;
  uint32_t k;            // elements kept by top-k (V: all)
  uint32_t p24, least;   // top-p as a multiple of 2^-24; min-p's smallest weight
  uint32_t u31;
  bool need_k, need_p;
};

__device__ __forceinline__ float logp_of(const Filter& f, float z, uint64_t total) {
  return __fsub_rn(__fdiv_rn(__fsub_rn(z, f.m), f.tau),
                   logf(__fmul_rn(__ull2float_rn(total), 0x1p-31f)));
}

// The leading CTA's end of a row whose cut lies within the n listed candidates (all of the
// row's elements up to some place in the sorted order): sort them, cut, and take the token.
__device__ __forceinline__ void finish_list(const Block& b, const Filter& f, const SampleArgs& a,
                                            int row, int n, uint64_t total_mass) {
  SampleSmem* s = b.s;
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kSampleThreads) s->list[i] = ~0ull;
  __syncthreads();
  block_sort(s->list, size);
  // by descending logit: thread t takes the t-th run of `each` candidates
  const int each = size > kSampleThreads ? size / kSampleThreads : 1;
  const int i0 = threadIdx.x * each;
  uint32_t w[kList / kSampleThreads];
  uint64_t sum = 0;
  uint32_t zero = 0;
#pragma unroll
  for (int e = 0; e < kList / kSampleThreads; ++e) {
    w[e] = 0;
    if (e < each && i0 + e < n && (uint32_t)(i0 + e) < f.k)
      w[e] = weight_of(x_of(logit_of(~(uint32_t)(s->list[i0 + e] >> 32)), f.m, f.c));
    sum += w[e];
  }
  uint64_t upto = sum;
  block_scan(b, zero, upto);
  if (threadIdx.x == kSampleThreads - 1) s->part[5][0] = upto;
  __syncthreads();
  uint64_t most = f.need_k ? s->part[5][0] : total_mass;    // C_k
  most = scaled_24(most, f.p24);
  if (most < 1) most = 1;
  uint64_t before = upto - sum;
  uint64_t entry[kList / kSampleThreads];
#pragma unroll
  for (int e = 0; e < kList / kSampleThreads; ++e) {
    if (e < each && i0 + e < size) {
      const uint32_t keep = before < most && w[e] >= f.least ? w[e] : 0;
      entry[e] = i0 + e < n ? (s->list[i0 + e] << 32) | keep : ~0ull;   // (id, weight)
    }
    before += w[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kList / kSampleThreads; ++e)
    if (e < each && i0 + e < size) s->list[i0 + e] = entry[e];
  __syncthreads();
  block_sort(s->list, size);                                // by id
  sum = 0;
#pragma unroll
  for (int e = 0; e < kList / kSampleThreads; ++e) {
    w[e] = e < each && i0 + e < n ? (uint32_t)s->list[i0 + e] : 0;
    sum += w[e];
  }
  upto = sum;
  block_scan(b, zero, upto);
  if (threadIdx.x == kSampleThreads - 1) s->part[5][1] = upto;
  __syncthreads();
  const uint64_t total = s->part[5][1];
  const uint64_t at = scaled_31(total, f.u31);
  before = upto - sum;
#pragma unroll
  for (int e = 0; e < kList / kSampleThreads; ++e) {
    if (before <= at && at < before + w[e]) {
      const int id = (int)(s->list[i0 + e] >> 32);
      if (RLK_STORE_OK(row < a.N && id >= 0 && id < a.V, &g_err_sample)) {
        a.token[row] = id;
        s->answer = id;
      }
    }
    before += w[e];
  }
  if (threadIdx.x == 0) s->xmass[3] = total;
}

template <bool kFp32>
__global__ void __launch_bounds__(kSampleThreads, 2)
    sample_kernel(SampleArgs a, int per) {
  using R = Row<kFp32>;
  constexpr int kE = R::kElems;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem* s = reinterpret_cast<SampleSmem*>(smem_raw);
  uint4* vecs = reinterpret_cast<uint4*>(smem_raw + sizeof(SampleSmem));
  Block b;
  b.s = s;
  b.rank = (int)cluster_rank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(b.ctas));
  const int row = blockIdx.x / b.ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s->n_list = 0;
  griddep_wait();
  if (tid == 0) griddep_launch_dependents();

  // ---- settings of the row
  Filter f;
  float tau = a.temperature ? __ldg(a.temperature + row) : a.temperature_all;
  int k = a.top_k ? __ldg(a.top_k + row) : a.top_k_all;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : a.top_p_all;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : a.min_p_all;
  const double u = a.uniform_fp64 ? __ldg(static_cast<const double*>(a.uniform) + row)
                                  : (double)__ldg(static_cast<const float*>(a.uniform) + row);
  bool bad = !(tau >= 0.f && tau < INFINITY) || top_p != top_p || min_p != min_p || u != u;
  if (tau < 1e-6f) {
    tau = 1.f;
    k = 1;
  }
  f.tau = tau;
  f.c = __fdiv_rn(kLog2e, tau);
  f.k = k > 0 && k < a.V ? (uint32_t)k : (uint32_t)a.V;
  f.need_k = f.k < (uint32_t)a.V;
  f.p24 = (uint32_t)rintf(__fmul_rn(fminf(fmaxf(top_p, 0.f), 1.f), 16777216.f));
  f.need_p = f.p24 < (1u << 24);
  f.least = (uint32_t)rintf(__fmul_rn(fminf(fmaxf(min_p, 0.f), 1.f), 16777216.f)) << 7;
  f.u31 = (uint32_t)fmin(fmax(floor(u * 2147483648.0), 0.0), 2147483647.0);

  // ---- the row into shared memory, and its maximum
  const int esize = kFp32 ? 4 : 2;
  const uintptr_t start = reinterpret_cast<uintptr_t>(a.logits) + (uintptr_t)(row * a.ld) * esize;
  const int lead = (int)(start & 15) / esize;
  const uint4* src = reinterpret_cast<const uint4*>(start & ~(uintptr_t)15);
  const int vectors = (lead + a.V + kE - 1) / kE;
  const int cta0 = b.rank * per;
  const int mine = max(0, min(per, vectors - cta0));
  R r;
  r.smem = vecs;
  r.first_id = cta0 * kE - lead;
  const int each = (mine + kSampleWarps - 1) / kSampleWarps;
  r.v0 = min(warp * each, mine);
  r.v1 = min(r.v0 + each, mine);
  float top = -INFINITY;
#pragma unroll 4
  for (int v = r.v0 + lane; v < r.v1; v += 32) {
    const int id0 = r.first_id + v * kE;
    uint4 q;
    if (id0 >= 0 && id0 + kE <= a.V) {
      q = __ldg(src + cta0 + v);
    } else {                                       // the row's first or last vector, in part
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kFp32) {
          p[i] = 0xff800000u;
          if (id0 + i >= 0 && id0 + i < a.V)
            p[i] = __ldg(reinterpret_cast<const uint32_t*>(start) + id0 + i);
        } else {
          uint32_t h[2] = {0xff80u, 0xff80u};
#pragma unroll
          for (int o = 0; o < 2; ++o)
            if (id0 + 2 * i + o >= 0 && id0 + 2 * i + o < a.V)
              h[o] = __ldg(reinterpret_cast<const uint16_t*>(start) + id0 + 2 * i + o);
          p[i] = h[0] | (h[1] << 16);
        }
      }
      q = make_uint4(p[0], p[1], p[2], p[3]);
    }
    vecs[v] = q;
    float z[kE];
    R::unpack(q, z);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      bad |= !(z[e] < INFINITY);                   // NaN or +inf
      top = fmaxf(top, z[e]);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  bad = __any_sync(kFull, bad);
  if (lane == 0) s->part[0][warp] = ((uint64_t)bad << 32) | key_of(top);
  __syncthreads();
  if (tid == 0) {
    uint64_t v = 0;                                // a bad part outranks any logit
    for (int w = 0; w < kSampleWarps; ++w) v = max(v, s->part[0][w]);
    s->xch[0] = v;
  }
  cluster_join();
  {
    uint64_t v = 0;
    for (int i = 0; i < b.ctas; ++i) v = max(v, ld_cluster_u64(b.peer(&s->xch[0], i)));
    f.m = logit_of((uint32_t)v);
    bad = (v >> 32) != 0 || f.m == -INFINITY;
  }
  if (bad) {                                       // nothing to draw from
    if (b.rank == 0 && tid == 0 && RLK_STORE_OK(row < a.N, &g_err_sample)) {
      a.token[row] = -1;
      a.logp[row] = __int_as_float(0x7fc00000);
    }
    cluster_join();                                // peers may still read this CTA's value
    return;
  }

  // ---- where the kept prefix of the sorted order ends: key > cut_key, or equal and id <= cut_id
  uint32_t cut_key = 0;
  int cut_id = a.V;
  bool by_mass = !f.need_k;                        // the search under way
  uint64_t total_mass = 0, want_mass = 0;
  uint32_t want_count = f.k;
  int slot = 1;
  // at most: by count, by weight instead if that cuts nothing, or by weight after it
  for (int pass = 0; pass < 2 && (f.need_k || f.need_p); ++pass) {
    Cut cut;
    uint32_t before = 0;                           // elements, weight above the current range
    uint64_t mass_before = 0;
    int window = 0;
    for (; window < kWindows; ++window) {
      clear_bins(b, f.need_p);
      uint64_t mass = 0;
      for (int v = r.v0 + lane; v < r.v1; v += 32) {
        float z[kE];
        r.get(v, z);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float x = x_of(z[e], f.m, f.c);
          const int bin = bin_of(x, window);
          uint32_t w = 0;
          if (f.need_p) {
            w = weight_of(x);
            mass += w;
          }
          if (bin >= 0 && bin < kBins) add_to_bin(b, bin, f.need_p, w);
        }
      }
      if (by_mass && window == 0 && total_mass == 0) {   // C_k is the whole row's weight
        mass = block_sum(b, mass, 1);
        if (tid == 0) s->xmass[0] = mass;
        cluster_join();
        for (int i = 0; i < b.ctas; ++i) total_mass += ld_cluster_u64(b.peer(&s->xmass[0], i));
        want_mass = scaled_24(total_mass, f.p24);
        if (want_mass < 1) want_mass = 1;
      }
      uint32_t all_n;
      uint64_t all_mass;
      cut = find_cut(b, f.need_p, by_mass, want_count - before, want_mass - mass_before, &all_n,
                     &all_mass);
      if (cut.bin >= 0) break;
      before += all_n;
      mass_before += all_mass;
    }
    if (cut.bin < 0) {
      // Only weightless elements are left: top-k cuts nothing that could be drawn.
      if (f.need_k && f.need_p && !by_mass) {
        f.need_k = false;
        by_mass = true;
        continue;
      }
      break;
    }
    const bool first = f.need_k == !by_mass;       // the search that any list would end
    before += cut.before;
    mass_before += cut.mass;
    if (first && before + cut.in <= kList) {
      // ---- few candidates: the leading CTA takes them all
      for (int v = r.v0 + lane; v < r.v1; v += 32) {
        float z[kE];
        r.get(v, z);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          if (bin_of(x_of(z[e], f.m, f.c), window) <= cut.bin) {
            const uint32_t at = atom_add_cluster(b.peer(&s->n_list, 0), 1);
            if (at < kList)
              st_cluster_u64(b.peer(&s->list[at], 0),
                             ((uint64_t)~key_of(z[e]) << 32) | (uint32_t)(r.first_id + v * kE + e));
          }
        }
      }
      cluster_join();
      if (b.rank == 0) {
        const int n = (int)(before + cut.in);
        finish_list(b, f, a, row, n, total_mass);
        __syncthreads();
        if (tid == 0 && RLK_STORE_OK(row < a.N, &g_err_sample)) {
          const int id = s->answer;
          const float z =
              kFp32 ? __ldg(static_cast<const float*>(a.logits) + row * a.ld + id)
                    : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.logits) +
                                                      row * a.ld + id)
                                      << 16);
          a.logp[row] = logp_of(f, z, s->xmass[3]);
        }
      }
      return;
    }
    // ---- narrow the cut inside the bin: first the bin's range of keys ...
    uint32_t kmin = 0xffffffffu, kmax = 0;
    for (int v = r.v0 + lane; v < r.v1; v += 32) {
      float z[kE];
      r.get(v, z);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (bin_of(x_of(z[e], f.m, f.c), window) == cut.bin) {
          kmin = min(kmin, key_of(z[e]));
          kmax = max(kmax, key_of(z[e]));
        }
    }
    kmin = __reduce_min_sync(kFull, kmin);
    kmax = __reduce_max_sync(kFull, kmax);
    __syncthreads();
    if (lane == 0) s->part[2][warp] = ((uint64_t)~kmin << 32) | kmax;
    __syncthreads();
    if (tid == 0) {
      uint32_t lo = 0, hi = 0;
      for (int w = 0; w < kSampleWarps; ++w) {
        lo = max(lo, (uint32_t)(s->part[2][w] >> 32));
        hi = max(hi, (uint32_t)s->part[2][w]);
      }
      s->xch[slot] = ((uint64_t)lo << 32) | hi;
    }
    cluster_join();
    {
      uint32_t lo = 0, hi = 0;
      for (int i = 0; i < b.ctas; ++i) {
        const uint64_t v = ld_cluster_u64(b.peer(&s->xch[slot], i));
        lo = max(lo, (uint32_t)(v >> 32));
        hi = max(hi, (uint32_t)v);
      }
      kmin = ~lo;
      kmax = hi;
    }
    ++slot;
    // ... then that range in kBins parts until a part is one key
    uint32_t in = cut.in;
    for (int level = 0; kmin != kmax && level < 4; ++level) {   // 32 bits, 10 a level
      int shift = 0;
      while (((kmax - kmin) >> shift) >= kBins) ++shift;
      clear_bins(b, f.need_p);
      for (int v = r.v0 + lane; v < r.v1; v += 32) {
        float z[kE];
        r.get(v, z);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const uint32_t key = key_of(z[e]);
          if (key >= kmin && key <= kmax)
            add_to_bin(b, (kmax - key) >> shift, f.need_p,
                       f.need_p ? weight_of(x_of(z[e], f.m, f.c)) : 0);
        }
      }
      uint32_t all_n;
      uint64_t all_mass;
      cut = find_cut(b, f.need_p, by_mass, want_count - before, want_mass - mass_before, &all_n,
                     &all_mass);
      before += cut.before;
      mass_before += cut.mass;
      in = cut.in;
      const uint32_t hi = kmax - ((uint32_t)cut.bin << shift);
      const uint32_t below = (1u << shift) - 1;
      kmin = hi - kmin > below ? hi - below : kmin;
      kmax = hi;
    }
    cut_key = kmax;
    const uint32_t w = weight_of(x_of(logit_of(cut_key), f.m, f.c));
    uint64_t keep;                                 // how many of the equal ones
    if (by_mass)
      keep = w ? (want_mass - mass_before + w - 1) / w : in;
    else
      keep = want_count - before;
    if (keep > in) keep = in;
    if (!by_mass && f.need_p) {                    // top-p among the k kept
      total_mass = mass_before + keep * w;
      want_mass = scaled_24(total_mass, f.p24);
      if (want_mass < 1) want_mass = 1;
      by_mass = true;
      continue;
    }
    if (keep < in) {
      // ---- the id of the keep-th equal logit
      uint32_t ties = 0;
      for (int v = r.v0 + lane; v < r.v1; v += 32) {
        float z[kE];
        r.get(v, z);
#pragma unroll
        for (int e = 0; e < kE; ++e) ties += key_of(z[e]) == cut_key;
      }
      ties = __reduce_add_sync(kFull, ties);
      __syncthreads();
      if (lane == 0) s->part[3][warp] = ties;
      __syncthreads();
      uint64_t below = 0, here = 0;                // ties in earlier CTAs; in this CTA's earlier warps
      for (int w2 = 0; w2 < kSampleWarps; ++w2) here += s->part[3][w2];
      if (tid == 0) s->xch[slot] = here;
      cluster_join();
      for (int i = 0; i < b.rank; ++i) below += ld_cluster_u64(b.peer(&s->xch[slot], i));
      ++slot;
      for (int w2 = 0; w2 < warp; ++w2) below += s->part[3][w2];
      if (tid == 0) s->xch[slot] = 0;
      __syncthreads();
      if (below < keep && keep <= below + ties) {  // uniform in the warp: its part holds it
        for (int v = r.v0; v < r.v1; v += 32) {
          float z[kE];
          uint32_t n = 0;
          if (v + lane < r.v1) {
            r.get(v + lane, z);
#pragma unroll
            for (int e = 0; e < kE; ++e) n += key_of(z[e]) == cut_key;
          }
          uint32_t upto = n;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(kFull, upto, off);
            if (lane >= off) upto += o;
          }
          const uint64_t prior = below + upto - n;
          if (prior < keep && keep <= below + upto) {
            uint64_t seen = prior;
            for (int e = 0; e < kE; ++e)
              if (key_of(z[e]) == cut_key && ++seen == keep)
                s->xch[slot] = (uint32_t)(r.first_id + (v + lane) * kE + e) + 1u;
          }
          below += __shfl_sync(kFull, upto, 31);
        }
      }
      cluster_join();
      uint64_t id = 0;
      for (int i = 0; i < b.ctas; ++i) id = max(id, ld_cluster_u64(b.peer(&s->xch[slot], i)));
      ++slot;
      cut_id = (int)id - 1;
    }
    break;
  }

  // ---- weights kept, by warp and CTA
  uint64_t sum = 0;
  for (int v = r.v0 + lane; v < r.v1; v += 32) {
    float z[kE];
    r.get(v, z);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const uint32_t key = key_of(z[e]);
      if (key > cut_key || (key == cut_key && r.first_id + v * kE + e <= cut_id)) {
        const uint32_t w = weight_of(x_of(z[e], f.m, f.c));
        if (w >= f.least) sum += w;
      }
    }
  }
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s->part[0][warp] = sum;
  __syncthreads();
  uint64_t here = 0, before = 0, total = 0;
  for (int w = 0; w < kSampleWarps; ++w) here += s->part[0][w];
  if (tid == 0) s->xmass[1] = here;
  cluster_join();
  for (int i = 0; i < b.ctas; ++i) {
    const uint64_t v = ld_cluster_u64(b.peer(&s->xmass[1], i));
    if (i < b.rank) before += v;
    total += v;
  }
  for (int w = 0; w < warp; ++w) before += s->part[0][w];
  const uint64_t at = scaled_31(total, f.u31);
  if (before <= at && at < before + sum) {         // uniform in the warp: the token is in its part
    for (int v = r.v0; v < r.v1; v += 32) {
      float z[kE];
      uint32_t w[kE];
      uint64_t n = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] = 0;
      if (v + lane < r.v1) {
        r.get(v + lane, z);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const uint32_t key = key_of(z[e]);
          if (key > cut_key || (key == cut_key && r.first_id + (v + lane) * kE + e <= cut_id)) {
            w[e] = weight_of(x_of(z[e], f.m, f.c));
            if (w[e] < f.least) w[e] = 0;
          }
          n += w[e];
        }
      }
      uint64_t upto = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t o = __shfl_up_sync(kFull, upto, off);
        if (lane >= off) upto += o;
      }
      uint64_t prior = before + upto - n;
      if (prior <= at && at < before + upto) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          if (prior <= at && at < prior + w[e]) {
            const int id = r.first_id + (v + lane) * kE + e;
            if (RLK_STORE_OK(row < a.N && id >= 0 && id < a.V, &g_err_sample)) {
              a.token[row] = id;
              a.logp[row] = logp_of(f, z[e], total);
            }
          }
          prior += w[e];
        }
      }
      before += __shfl_sync(kFull, upto, 31);
    }
  }
  cluster_join();                                  // peers have read this CTA's sum
}

std::mutex g_attr_mutex;
bool g_attr_set[64];

cudaError_t ensure_attrs(int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_attr_set[dev]) return cudaSuccess;
  for (auto* kernel : {sample_kernel<false>, sample_kernel<true>}) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  g_attr_set[dev] = true;
  return cudaSuccess;
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// CTAs a row: enough that a CTA holds at most 76 KiB of it (two CTAs fit an SM), then
// doubled while the clusters leave SMs idle and a CTA keeps 2 Ki elements or more.
int cluster_ctas(int64_t N, int64_t V, int esize, int sms) {
  int c = 1;
  while (c < kMaxCluster && ceil_div(V, c) * esize > 77824) c *= 2;
  while (c < kMaxCluster && N * c * 2 <= sms && V / (2 * c) >= 2048) c *= 2;
  return c;
}

}  // namespace

uint32_t take_error_sample() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_sample, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaMemcpyToSymbol(g_err_sample, &zero, sizeof zero);
  cudaGetLastError();
  return v;
}

}  // namespace rlk

using namespace rlk;

extern "C" rlk_status rlk_sample_logits(const void* logits, int logits_dtype, int64_t N, int64_t V,
                                        int64_t ld, const void* uniform, int uniform_dtype,
                                        const float* temperature, float temperature_all,
                                        const int32_t* top_k, int32_t top_k_all,
                                        const float* top_p, float top_p_all, const float* min_p,
                                        float min_p_all, int64_t* token, float* logp,
                                        void* stream) {
  RLK_CALL_RANGE();
  if (N < 0 || N >= (int64_t(1) << 27) || V < 1 || V > kMaxSampleVocab || ld < V ||
      ld >= (int64_t(1) << 36))
    return RLK_ERR_SHAPE;
  if ((logits_dtype != RLK_BF16 && logits_dtype != RLK_FP32) ||
      (uniform_dtype != RLK_FP32 && uniform_dtype != RLK_FP64))
    return RLK_ERR_DTYPE;
  if ((!temperature && !(temperature_all >= 0.f && temperature_all < INFINITY)) ||
      (!top_p && top_p_all != top_p_all) || (!min_p && min_p_all != min_p_all))
    return RLK_ERR_VALUE;
  if (N == 0) return RLK_OK;
  if (!logits || !uniform || !token || !logp) return RLK_ERR_NULL;
  const bool fp32 = logits_dtype == RLK_FP32;
  if (!aligned_to(logits, fp32 ? 4 : 2) || !aligned_to(uniform, uniform_dtype == RLK_FP64 ? 8 : 4) ||
      !aligned_to(temperature, 4) || !aligned_to(top_k, 4) || !aligned_to(top_p, 4) ||
      !aligned_to(min_p, 4) || !aligned_to(token, 8) || !aligned_to(logp, 4))
    return RLK_ERR_ALIGN;
  DeviceInfo dev;
  const rlk_status st = device_ready(&dev);
  if (st != RLK_OK) return st;
  if (ensure_attrs(dev.device) != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  SampleArgs a;
  a.logits = logits;
  a.ld = ld;
  a.N = (int)N;
  a.V = (int)V;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.temperature_all = temperature_all;
  a.top_k_all = top_k_all;
  a.top_p_all = top_p_all;
  a.min_p_all = min_p_all;
  a.uniform = uniform;
  a.uniform_fp64 = uniform_dtype == RLK_FP64;
  a.token = token;
  a.logp = logp;
  const int ctas = cluster_ctas(N, V, fp32 ? 4 : 2, dev.sm_count);
  const int elems = fp32 ? 4 : 8;
  // vectors of a row that starts anywhere in its first vector, dealt evenly
  const int per = (int)ceil_div(ceil_div(V + elems - 1, elems), ctas);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * ctas));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = sizeof(SampleSmem) + (size_t)per * 16;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = fp32 ? cudaLaunchKernelEx(&cfg, sample_kernel<true>, a, per)
                             : cudaLaunchKernelEx(&cfg, sample_kernel<false>, a, per);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return RLK_OK;
}
