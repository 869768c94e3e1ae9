// Building blocks of the sampling kernels (sample.cu): weights as whole numbers, a row's
// vectors, what the CTAs of a cluster exchange, histograms and where they are cut, lists of
// candidates and how a row ends from one.  Included by sample.cu alone.
#pragma once

#include <math.h>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_pipeline.cuh"

namespace rlk {

__device__ unsigned int g_err_sample = 0;

namespace {

constexpr int kMaxSampleWarps = 32;
constexpr int kBins = 1024;                  // histogram bins
constexpr int kList = 2048;                  // candidates the leading CTA sorts
constexpr int kMaxCluster = 16;
constexpr int64_t kMaxSampleVocab = 524288;
constexpr int64_t kMaxSampleRows = int64_t(1) << 20;
constexpr float kOctaves = 32.f;             // weights vanish below 2^-32
constexpr float kNear = 20.f;                // octaves of top-p's first histogram
constexpr uint32_t kOne = 1u << 31;
constexpr uint32_t kFull = 0xffffffffu;

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
  int fp32;
  int64_t* token;
  float* logp;
  const int* left;            // not null: their number and the rows to take, of all
};

// ---------------------------------------------------------------- weights
__device__ __forceinline__ float x_of(float z, float m, float c) {
  return fmaxf(__fmul_rn(__fsub_rn(z, m), c), -126.f);
}

// Two weights, 2^(x + 31) rounded to a whole number (nearest even), from two logits.  The
// packed operations round each half as the single ones do.  x + 1.5 2^23 rounds x to a
// whole number n and leaves it in the low bits; the polynomial's coefficients carry the
// factor 2^31, and n is added to the result's exponent.
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t both(float a) { return pack_f2(a, a); }

// A product that stays rounded by itself: written as mul.rn.f32x2, the assembler merges it with
// a sum that follows into one fused operation, rounding once (the single mul.rn.f32 is left
// alone).  a * b + -0 is the rounded product, signed zeros included; the -0 is read from memory
// that a host may write, so that nothing can be folded.
__constant__ float g_minus_zero = -0.f;
__device__ __forceinline__ uint64_t mul_alone_f2(uint64_t a, uint64_t b, uint64_t minus_zero) {
  return fma_f2(a, b, minus_zero);
}

constexpr float kRound = 12582912.f;         // 1.5 * 2^23

__device__ __forceinline__ void weights_of(float x0, float x1, uint32_t& w0, uint32_t& w1) {
  constexpr float kExp2[6] = {0.0013264727313071489f * 0x1p31f, 0.009671512991189957f * 0x1p31f,
                              0.05550733581185341f * 0x1p31f, 0.24022242426872253f * 0x1p31f,
                              0.6931470036506653f * 0x1p31f, 0x1p31f};
  const uint64_t x = pack_f2(x0, x1);
  const uint64_t t = add_f2(x, both(kRound));
  const uint64_t n = add_f2(t, both(-kRound));
  const uint64_t f = fma_f2(n, both(-1.f), x);     // x - n, exact
  const uint64_t minus_zero = both(g_minus_zero);
  uint64_t y = both(kExp2[0]);
#pragma unroll
  for (int i = 1; i < 6; ++i) y = add_f2(mul_alone_f2(y, f, minus_zero), both(kExp2[i]));
  float t0, t1, y0, y1;
  unpack_f2(t, t0, t1);
  unpack_f2(y, y0, y1);
  w0 = __float2uint_rn(__int_as_float(__float_as_int(y0) + (__float_as_int(t0) << 23)));
  w1 = __float2uint_rn(__int_as_float(__float_as_int(y1) + (__float_as_int(t1) << 23)));
}
// x of two logits, by the operations of x_of.
__device__ __forceinline__ void x_pair(float z0, float z1, float m, float c, float& x0, float& x1) {
  unpack_f2(mul_f2(add_f2(pack_f2(z0, z1), both(-m)), both(c)), x0, x1);
  x0 = fmaxf(x0, -126.f);
  x1 = fmaxf(x1, -126.f);
}
__device__ __forceinline__ uint32_t weight_of(float x) {
  uint32_t w, unused;
  weights_of(x, x, w, unused);
  return w;
}

// a + b as one multiply-add.
__device__ __forceinline__ uint64_t add_wide(uint64_t a, uint32_t b) {
  uint64_t v;
  asm("mad.wide.u32 %0, %1, 1, %2;" : "=l"(v) : "r"(b), "l"(a));
  return v;
}

// Order-preserving bit pattern of a logit (+0 and -0 alike).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.f));
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// A range of octaves below the top, and the bin of x in it, 0 .. kBins - 1.  The bin falls
// with x, so a bin is a run of the sorted order.
struct Window {
  float from, to, scale, origin;
  __device__ __forceinline__ Window(float from, float to)
      : from(from), to(to), scale((kBins - 1) / (to - from)), origin(kRound - from * scale) {}
  // for x in [-to, -from]
  __device__ __forceinline__ int at(float x) const {
    return __float_as_int(__fmaf_rn(x, -scale, origin)) - __float_as_int(kRound);
  }
  __device__ __forceinline__ bool has(float x) const { return x > -to && x <= -from; }
  // -1 above the range, kBins below it
  __device__ __forceinline__ int bin(float x) const {
    return x <= -to ? kBins : (x > -from ? -1 : at(x));
  }
};
__device__ __forceinline__ Window all_octaves() { return Window(0.f, kOctaves); }

// floor(a b / 2^31) and floor(a p / 2^24), a < 2^50, b < 2^31, p <= 2^24, exactly.
__device__ __forceinline__ uint64_t scaled_31(uint64_t a, uint32_t b) {
  return (a >> 31) * b + (((a & (kOne - 1)) * b) >> 31);
}
__device__ __forceinline__ uint64_t scaled_24(uint64_t a, uint32_t p) {
  return (((a >> 31) * p) << 7) + (((a & (kOne - 1)) * p) >> 24);
}

// A load that stays where it stands (an ordinary one sinks to its use, behind a condition,
// and the loads of a batch go out one after another's return).
__device__ __forceinline__ uint4 load_now(const uint4* p) {
  uint4 q;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// ---------------------------------------------------------------- the row
// The row in 16-byte vectors of its memory: element j of the vectors is id j - lead, where
// lead (< one vector) is how far the row's start lies past a 16-byte boundary; elements
// outside the row are -inf.  The CTA of rank r has vectors [r * per, (r + 1) * per); in
// every pass, warp w takes a contiguous part of them, a vector per lane and step, so the
// order (CTA, warp, step, lane, element) is the order of ids.
template <bool kFp32, bool kOnChip>
struct Row {
  static constexpr int kElems = kFp32 ? 4 : 8;
  const uint4* memory;   // the CTA's first vector in global memory
  uint4* chip;           // and in shared memory
  const void* start;     // id 0
  int first_id;          // id of the CTA's element 0
  int V;
  int full0, full1;      // the CTA's vectors that lie in the row as a whole
  int v0, v1;            // this warp's vectors, from the CTA's first

  // Sets all but chip, v0 and v1 for the row's vectors; returns their number.
  __device__ __forceinline__ int begin(const SampleArgs& a, int row) {
    const int esize = kFp32 ? 4 : 2;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) + (uintptr_t)(row * a.ld) * esize;
    const int lead = (int)(at & 15) / esize;
    memory = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
    chip = nullptr;
    start = reinterpret_cast<const void*>(at);
    first_id = -lead;
    V = a.V;
    full0 = lead > 0 ? 1 : 0;
    full1 = (lead + a.V) / kElems;
    return (lead + a.V + kElems - 1) / kElems;
  }
  // Counts vectors from the n-th on.
  __device__ __forceinline__ void skip(int n) {
    memory += n;
    first_id += n * kElems;
    full0 -= n;
    full1 -= n;
  }
  __device__ __forceinline__ int id_of(int v) const { return first_id + v * kElems; }
  __device__ __forceinline__ bool whole(int v) const { return v >= full0 && v < full1; }
  __device__ __forceinline__ uint4 load_part(int v) const {
    const int id0 = id_of(v);                      // the row's first or last vector
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kFp32) {
        p[i] = 0xff800000u;
        if (id0 + i >= 0 && id0 + i < V) p[i] = __ldg(static_cast<const uint32_t*>(start) + id0 + i);
      } else {
        uint32_t h[2] = {0xff80u, 0xff80u};
#pragma unroll
        for (int o = 0; o < 2; ++o)
          if (id0 + 2 * i + o >= 0 && id0 + 2 * i + o < V)
            h[o] = __ldg(static_cast<const uint16_t*>(start) + id0 + 2 * i + o);
        p[i] = h[0] | (h[1] << 16);
      }
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ uint4 get(int v) const {
    if constexpr (kOnChip) return chip[v];
    return whole(v) ? __ldg(memory + v) : load_part(v);
  }
  // Several vectors, all on their way before any is used: the loads are unconditional (of
  // some whole vector where v is not one), and the row's ends are set right afterwards.
  template <bool kFromMemory, int kN>
  __device__ __forceinline__ void get_all(const int (&v)[kN], uint4 (&q)[kN]) const {
    if constexpr (kOnChip && !kFromMemory) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (v[i] < v1) q[i] = chip[v[i]];
    } else {
      if (full1 > full0) {
#pragma unroll
        for (int i = 0; i < kN; ++i) q[i] = load_now(memory + min(max(v[i], full0), full1 - 1));
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (!whole(v[i]) && v[i] < v1) q[i] = load_part(v[i]);
    }
  }
  // The warp's vectors in order, kN a lane at a time: use(vector, its elements).
  template <bool kFromMemory, int kN, class F>
  __device__ __forceinline__ void each(F use) const {
    for (int base = v0; base < v1; base += 32 * kN) {
      int v[kN];
      uint4 q[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = base + 32 * i + (int)(threadIdx.x & 31);
      get_all<kFromMemory>(v, q);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (v[i] < v1) use(v[i], q[i]);
    }
  }
  __device__ __forceinline__ void get(int v, float (&z)[kElems]) const { unpack(get(v), z); }
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
  // Element t of an array of vectors.
  static __device__ __forceinline__ float element(const uint4* q, int t) {
    if constexpr (kFp32)
      return reinterpret_cast<const float*>(q)[t];
    else
      return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(q)[t] << 16);
  }
  // The largest of a vector's logits; NaN if one of them is.
  static __device__ __forceinline__ float top_of(const uint4& q) {
    float a, b;
    if constexpr (kFp32) {
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(__uint_as_float(q.x)), "f"(__uint_as_float(q.y)));
      asm("max.NaN.f32 %0, %1, %2, %3;"
          : "=f"(b)
          : "f"(__uint_as_float(q.z)), "f"(__uint_as_float(q.w)), "f"(a));
      return b;
    } else {
      uint32_t h, l;
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(h) : "r"(q.x), "r"(q.y));
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(l) : "r"(q.z), "r"(q.w));
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(l));
      asm("max.NaN.f32 %0, %1, %2;"
          : "=f"(a)
          : "f"(__uint_as_float(h << 16)), "f"(__uint_as_float(h & 0xffff0000u)));
      return a;
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
// Cluster barrier after code in which a warp's lanes may have parted.
__device__ __forceinline__ void cluster_join() {
  __syncwarp();
  cluster_sync();
}

struct Cut {             // where a search ended
  int bin;               // -1: nowhere in the histogram
  uint32_t before, in;   // elements in the bins before it, and in it
  uint64_t mass;         // weight of the bins before it
};

constexpr int kSlots = 10;

// Fixed shared memory; the row's vectors follow (kOnChip).  The list takes the histogram's
// place: it is filled after the second barrier of find_cut (or before any histogram), when
// no CTA reads another's histogram.
struct alignas(16) SampleSmem {
  union {
    struct {
      uint32_t count[kBins], lo[kBins], hi[kBins];   // this CTA's; weights as two halves
    };
    uint64_t list[kList];                        // this CTA's candidates; the leading CTA's, all
  };
  uint64_t slice_mass[kBins];                    // merged: this CTA's 1 / C of the bins
  uint32_t slice_count[kBins];
  // Values pushed here by the CTAs of the cluster, one set per exchange of the row.
  uint64_t from[kSlots][kMaxCluster];
  uint64_t part[4][kMaxSampleWarps];              // block reductions and scans
  uint64_t total[4];
  Cut cut;
  uint32_t top;                                  // this CTA's largest key
  uint32_t reached;                              // the least key that k threads' largest reach
  uint32_t n_list;                               // candidates of this CTA, listed or not
  uint32_t n_chunks;
  int answer;
};

static_assert(sizeof(SampleSmem) % 16 == 0, "the row's vectors follow, 16-byte aligned");

template <int kT>
struct Block {
  static constexpr int kThreads = kT, kWarps = kT / 32, kPerThread = kList / kT;
  SampleSmem* s;
  int rank, ctas;
  __device__ __forceinline__ uint32_t peer(const void* p, int r) const {
    return mapa_shared(smem_u32(p), (uint32_t)r);
  }
  // To every CTA of the cluster, this one included: from[slot][rank] = v.  The value of one
  // thread (warp 0 calls it); read after the next cluster barrier.
  __device__ __forceinline__ void push(int slot, uint64_t v) const {
    const int lane = threadIdx.x & 31;
    if (lane < ctas) st_cluster_u64(peer(&s->from[slot][rank], lane), v);
  }
  __device__ __forceinline__ uint64_t max_of(int slot) const {
    uint64_t v = 0;
    for (int i = 0; i < ctas; ++i) v = max(v, s->from[slot][i]);
    return v;
  }
  __device__ __forceinline__ uint64_t sum_of(int slot, int n) const {
    uint64_t v = 0;
    for (int i = 0; i < n; ++i) v += s->from[slot][i];
    return v;
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// Sum of v over the block, in warp 0 (the others' result is not used).
template <class B>
__device__ __forceinline__ uint64_t block_sum(const B& b, uint64_t v, int part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) b.s->part[part][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  if (threadIdx.x < B::kWarps) v = b.s->part[part][threadIdx.x];
  return threadIdx.x < 32 ? warp_sum(v) : 0;
}

// Inclusive prefix sums over the block's threads of (count, mass).
template <class B>
__device__ __forceinline__ void block_scan(const B& b, uint32_t& n, uint64_t& m) {
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
    b.s->part[2][warp] = n;
    b.s->part[3][warp] = m;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    n += (uint32_t)b.s->part[2][w];
    m += b.s->part[3][w];
  }
}

template <class B>
__device__ __forceinline__ void clear_bins(const B& b, bool mass) {
  for (int i = threadIdx.x; i < kBins; i += B::kThreads) {
    b.s->count[i] = 0;
    if (mass) {
      b.s->lo[i] = 0;
      b.s->hi[i] = 0;
    }
  }
  __syncthreads();
}

// 64-bit shared atomics are compare-and-swap loops (measured: 2 elements / ns / SM over
// scattered bins, 0.05 into one), 32-bit ones are not (5.8 and 0.9 for the three below).
template <class B>
__device__ __forceinline__ void add_to_bin(const B& b, int bin, bool mass, uint32_t w) {
  atomicAdd(&b.s->count[bin], 1u);
  if (mass) {
    atomicAdd(&b.s->lo[bin], w & 0xffffu);      // a CTA has fewer than 2^16 elements
    atomicAdd(&b.s->hi[bin], w >> 16);
  }
}

struct Filter {
  float m, c, tau;
  uint32_t k;            // elements kept by top-k (V: all)
  uint32_t p24, least;   // top-p as a multiple of 2^-24; min-p's smallest weight
  uint32_t u31;
  bool need_k, need_p;
  __device__ __forceinline__ uint32_t weight(float z) const { return weight_of(x_of(z, m, c)); }
  __device__ __forceinline__ uint64_t share(uint64_t mass) const {   // P
    const uint64_t v = scaled_24(mass, p24);
    return v < 1 ? 1 : v;
  }
};

// The first bin at which the running count reaches want_count, or (by_mass) the running
// weight reaches want_mass, over merged bins whose slices the CTAs of the cluster hold, after
// a barrier; *all_n and *all_mass are the whole count and weight.  s->cut.bin is -1 before.
template <class B>
__device__ __forceinline__ Cut scan_cut(const B& b, bool mass, bool by_mass, uint32_t want_count,
                                        uint64_t want_mass, uint32_t* all_n, uint64_t* all_mass) {
  SampleSmem* s = b.s;
  const int per = kBins / b.ctas;
  constexpr int kMine = kBins / B::kThreads;     // consecutive bins a thread
  const int bin = kMine * threadIdx.x;
  uint32_t n[kMine], cn = 0;
  uint64_t m[kMine], cm = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (b.ctas == 1) {
      n[i] = s->slice_count[bin + i];
      m[i] = mass ? s->slice_mass[bin + i] : 0;
    } else {
      const int owner = (bin + i) / per, at = (bin + i) - owner * per;
      n[i] = ld_cluster_u32(b.peer(&s->slice_count[at], owner));
      m[i] = mass ? ld_cluster_u64(b.peer(&s->slice_mass[at], owner)) : 0;
    }
    cn += n[i];
    cm += m[i];
  }
  uint32_t bn = cn;
  uint64_t bm = cm;
  block_scan(b, cn, cm);                         // inclusive, through this thread's bins
  bn = cn - bn;
  bm = cm - bm;
  if (threadIdx.x == B::kThreads - 1) {
    s->total[0] = cm;
    s->total[1] = cn;
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const bool was = by_mass ? bm >= want_mass : bn >= want_count;
    const bool is = by_mass ? bm + m[i] >= want_mass : bn + n[i] >= want_count;
    if (!was && is) s->cut = Cut{bin + i, bn, n[i], bm};
    bn += n[i];
    bm += m[i];
  }
  __syncthreads();
  *all_mass = s->total[0];
  *all_n = (uint32_t)s->total[1];
  return s->cut;
}

// After a cluster barrier that follows every CTA's histogram: merges them, and scan_cut.
template <class B>
__device__ __noinline__ Cut find_cut(B b, bool mass, bool by_mass,
                                        uint32_t want_count, uint64_t want_mass, uint32_t* all_n,
                                        uint64_t* all_mass) {
  SampleSmem* s = b.s;
  const int per = kBins / b.ctas;
  for (int i = threadIdx.x; i < per; i += B::kThreads) {
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
  return scan_cut(b, mass, by_mass, want_count, want_mass, all_n, all_mass);
}

// Ascending bitonic sort of n (a power of two, 64 or more) values in shared memory.  A warp
// does the steps within 64 values in registers; only longer steps go through shared memory.
__device__ __forceinline__ void order(uint64_t& x, uint64_t& y, bool up) {
  if ((x > y) == up) {
    const uint64_t t = x;
    x = y;
    y = t;
  }
}
template <class B>
__device__ __forceinline__ void block_sort(const B&, uint64_t* a, int n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int size = 64; size <= n; size <<= 1) {
    for (int step = size >> 1; step >= 64; step >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += B::kThreads) {
        const int i = 2 * t - (t & (step - 1));
        uint64_t x = a[i], y = a[i + step];
        order(x, y, (i & size) == 0);
        a[i] = x;
        a[i + step] = y;
      }
      __syncthreads();
    }
    for (int base = warp * 64; base < n; base += B::kWarps * 64) {
      uint64_t x = a[base + lane], y = a[base + 32 + lane];
      for (int part = size == 64 ? 2 : size; part <= size; part <<= 1) {
#pragma unroll
        for (int step = 32; step >= 1; step >>= 1) {
          if (step >= part) continue;
          if (step == 32) {
            order(x, y, ((base + lane) & part) == 0);
          } else {
            const bool low = (lane & step) == 0;
            const uint64_t ox = __shfl_xor_sync(kFull, x, step);
            const uint64_t oy = __shfl_xor_sync(kFull, y, step);
            const bool upx = ((base + lane) & part) == 0, upy = ((base + 32 + lane) & part) == 0;
            x = (low == upx) ? min(x, ox) : max(x, ox);
            y = (low == upy) ? min(y, oy) : max(y, oy);
          }
        }
      }
      a[base + lane] = x;
      a[base + 32 + lane] = y;
    }
    __syncthreads();
  }
}

// floor(u 2^31) of the row's uniform number, within [0, 2^31); all ones for a NaN.  An FP64
// number is taken by its bits: this GPU has little FP64 arithmetic.
__device__ __forceinline__ uint32_t uniform_31(const SampleArgs& a, int row) {
  if (!a.uniform_fp64) {
    const float u = __ldg(static_cast<const float*>(a.uniform) + row);
    return u != u ? kFull : min(__float2uint_rd(__fmul_rn(u, 0x1p31f)), kOne - 1);   // saturates
  }
  const uint64_t v = __ldg(static_cast<const unsigned long long*>(a.uniform) + row);
  const int e = (int)((v >> 52) & 0x7ff) - 1023;
  const uint64_t fraction = v & ((1ull << 52) - 1);
  if (e == 1024 && fraction) return kFull;
  if ((v >> 63) || e < -31) return 0;
  if (e >= 0) return kOne - 1;
  return (uint32_t)((fraction | (1ull << 52)) >> (21 - e));
}

// The row's settings (f.m is set later); *bad: they define no distribution.
__device__ __forceinline__ Filter settings_of(const SampleArgs& a, int row, bool* bad) {
  Filter f;
  f.m = 0.f;
  float tau = a.temperature ? __ldg(a.temperature + row) : a.temperature_all;
  int k = a.top_k ? __ldg(a.top_k + row) : a.top_k_all;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : a.top_p_all;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : a.min_p_all;
  f.u31 = uniform_31(a, row);
  *bad = !(tau >= 0.f && tau < INFINITY) || top_p != top_p || min_p != min_p || f.u31 == kFull;
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
  return f;
}

__device__ __forceinline__ void write_answer(const SampleArgs& a, const Filter& f, int row, int id,
                                             float z, uint64_t total) {
  if (RLK_STORE_OK(row < a.N && id >= 0 && id < a.V, &g_err_sample)) {
    a.token[row] = id;
    a.logp[row] = __fsub_rn(__fdiv_rn(__fsub_rn(z, f.m), f.tau),
                            logf(__fmul_rn(__ull2float_rn(total), 0x1p-31f)));
  }
}

// Candidate: sorts by descending logit, then by ascending id.
__device__ __forceinline__ uint64_t entry_of(float z, int id) {
  return ((uint64_t)~key_of(z) << 32) | (uint32_t)id;
}
__device__ __forceinline__ float entry_logit(uint64_t e) { return logit_of(~(uint32_t)(e >> 32)); }

template <class B>
__device__ __forceinline__ int sort_list(const B& b, int n) {
  SampleSmem* s = b.s;
  int size = 64;
  while (size < n) size <<= 1;
  if (n <= B::kThreads) {
    // An entry a thread, which counts those before it: no two are the same.
    const uint64_t mine = threadIdx.x < n ? s->list[threadIdx.x] : ~0ull;
    int rank = threadIdx.x;
    if (threadIdx.x < n) {
      rank = 0;
      int j = 0;
      for (; j + 4 <= n; j += 4) {
        const ulonglong2 x = reinterpret_cast<const ulonglong2*>(s->list)[j / 2];
        const ulonglong2 y = reinterpret_cast<const ulonglong2*>(s->list)[j / 2 + 1];
        rank += (x.x < mine) + (x.y < mine) + (y.x < mine) + (y.y < mine);
      }
      for (; j < n; ++j) rank += s->list[j] < mine;
    }
    __syncthreads();
    if (threadIdx.x < size) s->list[rank] = mine;
    __syncthreads();
    return size;
  }
  for (int i = n + threadIdx.x; i < size; i += B::kThreads) s->list[i] = ~0ull;
  __syncthreads();
  block_sort(b, s->list, size);
  return size;
}

// The end of a row of which the list holds all elements up to some place in the sorted
// order past the cut, n <= the block's threads, sorted: an element a thread.  One-off code is
// fetched as it runs, so it is kept short rather than unrolled (unrolled for one warp it took
// 5 us of a one-row call of 20).
template <class B>
__device__ __noinline__ void finish_short(B b, Filter f, const SampleArgs& a, int row, int n,
                                          uint64_t total_mass) {
  SampleSmem* s = b.s;
  const int i = threadIdx.x;
  const uint64_t x = s->list[min(i, n - 1)];
  const float z = entry_logit(x);
  const uint32_t id = (uint32_t)x;
  uint32_t w = i < n && (uint32_t)i < f.k ? f.weight(z) : 0, unused = 0;
  uint64_t upto = w;
  if (i == 0) s->answer = 0;
  block_scan(b, unused, upto);
  if (i == B::kThreads - 1) s->total[0] = upto;
  __syncthreads();
  const uint64_t most = f.share(f.need_k ? s->total[0] : total_mass);
  if (!(upto - w < most && w >= f.least)) w = 0;
  // A lower logit can have the larger weight, by a few units: min-p may drop one before another
  // that it keeps, so the places up to the last kept are taken, the dropped with no weight.
  if (i < n) s->list[i] = ((uint64_t)id << 32) | w;
  const int last = __reduce_max_sync(kFull, w ? i + 1 : 0);
  if ((i & 31) == 0) atomicMax(&s->answer, last);
  __syncthreads();
  const int kept = s->answer;
  if (i >= kept) return;
  uint64_t before = 0, total = 0;                  // kept weights of lower ids; of all
#pragma unroll 2
  for (int j = 0; j < kept; ++j) {
    const uint64_t o = s->list[j];
    total += (uint32_t)o;
    if ((uint32_t)(o >> 32) < id) before += (uint32_t)o;
  }
  const uint64_t at = scaled_31(total, f.u31);
  if (before <= at && at < before + w) write_answer(a, f, row, (int)id, z, total);
}

// The same for a longer list, by the block: sort by logit, cut, sort by id, take.
template <class B>
__device__ __forceinline__ void finish_block(const B& b, const Filter& f, const SampleArgs& a,
                                             int row, int n, int size, uint64_t total_mass) {
  SampleSmem* s = b.s;
  // thread t has the t-th run of `each` elements
  const int each = size > B::kThreads ? size / B::kThreads : 1;
  const int i0 = threadIdx.x * each;
  uint32_t w[B::kPerThread];
  uint64_t sum = 0;
  uint32_t unused = 0;
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    w[e] = 0;
    if (e < each && i0 + e < n && (uint32_t)(i0 + e) < f.k)
      w[e] = f.weight(entry_logit(s->list[i0 + e]));
    sum += w[e];
  }
  uint64_t upto = sum;
  block_scan(b, unused, upto);
  if (threadIdx.x == B::kThreads - 1) s->total[0] = upto;
  __syncthreads();
  const uint64_t most = f.share(f.need_k ? s->total[0] : total_mass);
  uint64_t before = upto - sum;
  uint64_t entry[B::kPerThread];
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    if (e < each && i0 + e < size) {
      const uint32_t keep = before < most && w[e] >= f.least ? w[e] : 0;
      entry[e] = i0 + e < n ? (s->list[i0 + e] << 32) | keep : ~0ull;   // (id, weight)
    }
    before += w[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e)
    if (e < each && i0 + e < size) s->list[i0 + e] = entry[e];
  __syncthreads();
  sort_list(b, n);                                          // by id
  sum = 0;
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    w[e] = e < each && i0 + e < n ? (uint32_t)s->list[i0 + e] : 0;
    sum += w[e];
  }
  upto = sum;
  block_scan(b, unused, upto);
  if (threadIdx.x == B::kThreads - 1) s->total[1] = upto;
  __syncthreads();
  const uint64_t total = s->total[1];
  const uint64_t at = scaled_31(total, f.u31);
  before = upto - sum;
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    if (before <= at && at < before + w[e]) s->answer = (int)(s->list[i0 + e] >> 32);
    before += w[e];
  }
  __syncthreads();
}

// The least logit whose bin (below the top m) is at most `bin` < kBins; the warp tries 32
// places of the range of keys at a time.  Every warp may call it by itself.  m is a number: from
// the key above all logits (NaN, +inf) the places would pass 2^32 and the search need not end.
__device__ __noinline__ float least_logit(float m, float c, Window window, int bin) {
  const int lane = threadIdx.x & 31;
  uint32_t no = key_of(-INFINITY), yes = key_of(m);
  while (yes - no > 1) {
    const uint32_t step = (yes - no) / 33 + 1;
    const uint32_t at = min(no + step * (lane + 1), yes);
    const uint32_t ok = __ballot_sync(kFull, window.bin(x_of(logit_of(at), m, c)) <= bin);
    const int first = ok ? __ffs(ok) - 1 : 32;     // ok is all ones from some lane on
    const uint32_t hi = first < 32 ? min(no + step * (first + 1), yes) : yes;
    no = min(no + step * first, yes - 1);
    yes = hi;
  }
  return logit_of(yes);
}

// Lists the elements of [lo, hi] among those of the warp's threads with `mine` set (the
// others have none).  Past the list's end they are only counted.  Where few threads have
// some, the warp shares their vectors out, so that all are on their way at once: a thread's
// own would be a chain of loads (512 rows of 151,936 from L2: 14 us a CTA for the chain).
template <class B, class R>
__device__ __forceinline__ void list_range(const B& b, const R& r, bool mine, float lo, float hi) {
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 31;
  const uint32_t who = __ballot_sync(kFull, mine);
  const int threads = __popc(who);
  const int steps = (r.v1 - r.v0 + 31) / 32;       // vectors a thread
  const bool share = threads <= 16;
  int at_rank = 0;                                 // the lane of the `lane`-th of them
#pragma unroll
  for (int step = 16; step >= 1; step >>= 1)
    if (__popc(who & ((1u << (at_rank + step)) - 1)) <= lane) at_rank += step;
  const int total = (share ? threads : 32) * steps;
  for (int i0 = 0; i0 < total; i0 += kBatch * 32) {
    uint4 q[kBatch];
    int v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = i0 + 32 * i + lane;
      int step = at >> 5, from = lane;
      if (share) {
        const int rank = at / steps;
        step = at - rank * steps;
        from = __shfl_sync(kFull, at_rank, rank & 31);
      }
      v[i] = at < total ? r.v0 + 32 * step + from : r.v1;
    }
    r.template get_all<false>(v, q);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (v[i] >= r.v1 || !(R::top_of(q[i]) >= lo)) continue;
      float z[R::kElems];
      R::unpack(q[i], z);
#pragma unroll
      for (int e = 0; e < R::kElems; ++e)
        if (z[e] >= lo && z[e] <= hi) {
          const uint32_t to = atomicAdd(&b.s->n_list, 1u);
          if (to < kList) b.s->list[to] = entry_of(z[e], r.id_of(v[i]) + e);
        }
    }
  }
}

template <class B, class R>
__device__ __noinline__ void list_range_cold(B b, R r, bool mine, float lo, float hi) {
  list_range(b, r, mine, lo, hi);
}

// After list_range: every CTA's count to all (read after the next cluster barrier).
template <class B>
__device__ __forceinline__ void push_count(const B& b) {
  __syncthreads();
  if (threadIdx.x < 32) b.push(7, b.s->n_list);
}

// The leading CTA appends the other CTAs' lists to its own; all leave together (the others
// must not before they have been read).  The sum of the counts is at most kList.
template <class B>
__device__ __forceinline__ void gather_lists(const B& b) {
  if (b.rank == 0 && b.ctas > 1) {
    const int lane = threadIdx.x & 31;
    int upto = lane < b.ctas ? (int)b.s->from[7][lane] : 0;   // entries of the CTAs up to this lane's
    const int mine = upto;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kFull, upto, off);
      if (lane >= off) upto += o;
    }
    const int n = __shfl_sync(kFull, upto, 31);
    for (int i0 = (int)b.s->from[7][0]; i0 < n; i0 += B::kThreads) {
      const int i = i0 + threadIdx.x;
      int r = 0;
      for (int c = 0; c < b.ctas; ++c) r += i >= __shfl_sync(kFull, upto, c);
      const int at = i - __shfl_sync(kFull, upto - mine, r & 31);
      if (i < n) b.s->list[i] = ld_cluster_u64(b.peer(&b.s->list[at], r));
    }
  }
  if (b.ctas > 1) cluster_join();
  __syncthreads();
}

// The smallest bin such that at least k threads' `bin` (kBins: none) do not exceed it;
// kBins - 1 where fewer than k threads have one.
__device__ __forceinline__ int reach_bin(int bin, uint32_t k) {
  int lo = 0;
#pragma unroll 1
  for (int step = kBins / 2; step >= 1; step >>= 1)
    if ((uint32_t)__syncthreads_count(bin < lo + step) < k) lo += step;
  return lo;
}

// Of the leading CTA's n listed candidates for top-k, keeps at least the k first, and few
// others: the threads' own best give a bin that the k first reach.
template <class B>
__device__ __forceinline__ int keep_first(const B& b, const Filter& f, int n) {
  SampleSmem* s = b.s;
  uint64_t entry[B::kPerThread];
  int bin[B::kPerThread], best = kBins;
#pragma unroll
  for (int i = 0; i < B::kPerThread; ++i) {
    const int at = i * B::kThreads + threadIdx.x;
    entry[i] = at < n ? s->list[at] : ~0ull;
    bin[i] = at < n ? all_octaves().bin(x_of(entry_logit(entry[i]), f.m, f.c)) : kBins;
    best = min(best, bin[i]);
  }
  __syncthreads();
  if (threadIdx.x == 0) s->n_list = 0;
  const int reach = reach_bin(best, f.k);          // its barriers order these accesses
#pragma unroll
  for (int i = 0; i < B::kPerThread; ++i)
    if (bin[i] <= reach) s->list[atomicAdd(&s->n_list, 1u)] = entry[i];
  __syncthreads();
  return (int)s->n_list;
}

// The leading CTA ends a row from its list of n elements.
template <class B>
__device__ __noinline__ void finish(B b, Filter f, const SampleArgs& a, int row, int n,
                                    uint64_t total_mass) {
  SampleSmem* s = b.s;
  // counting places is quadratic: 424 entries take 8 us, 60 take 1, and keep_first takes 2
  if (n > 96 && f.k <= B::kThreads) n = keep_first(b, f, n);
  const int size = sort_list(b, n);
  if (n <= B::kThreads) {
    finish_short(b, f, a, row, n, total_mass);
    return;
  }
  finish_block(b, f, a, row, n, size, total_mass);
  if (threadIdx.x == 0) {
    const int id = s->answer;
    const int64_t at = row * a.ld + id;
    const float z = a.fp32 ? __ldg(static_cast<const float*>(a.logits) + at)
                           : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.logits) +
                                                             at)
                                             << 16);
    write_answer(a, f, row, id, z, s->total[1]);
  }
}

// The leading CTA's search inside one bin, whose n elements it has listed: the last entry
// kept (s->total[2]) and the weight kept with it (s->total[3]).
template <class B>
__device__ __noinline__ void cut_in_bin(B b, Filter f, int n, bool by_mass,
                                           uint32_t keep, uint64_t mass_before,
                                           uint64_t want_mass) {
  SampleSmem* s = b.s;
  const int size = sort_list(b, n);
  const int each = size > B::kThreads ? size / B::kThreads : 1;
  const int i0 = threadIdx.x * each;
  uint32_t w[B::kPerThread];
  uint64_t sum = 0;
  uint32_t unused = 0;
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    w[e] = e < each && i0 + e < n ? f.weight(entry_logit(s->list[i0 + e])) : 0;
    sum += w[e];
  }
  uint64_t upto = sum;
  block_scan(b, unused, upto);
  uint64_t before = mass_before + upto - sum;
#pragma unroll
  for (int e = 0; e < B::kPerThread; ++e) {
    const bool last = by_mass ? before < want_mass && want_mass <= before + w[e]
                              : (uint32_t)(i0 + e) + 1 == keep;
    if (e < each && i0 + e < n && last) {
      s->total[2] = s->list[i0 + e];
      s->total[3] = before + w[e];
    }
    before += w[e];
  }
  __syncthreads();
}

// Adds the window's elements to the CTA's histogram with their weights; returns the weight
// of the thread's elements, of all of them (whole) or of some that include the window's.
template <class B, class R>
__device__ __noinline__ uint64_t weigh(B b, R r, float m, float c, Window window, bool whole) {
  constexpr int kE = R::kElems;
  uint64_t sum = 0;
  r.template each<false, 4>([&](int, const uint4& q) {
    const bool some = x_of(R::top_of(q), m, c) > -window.to;
    if (!(whole || some)) return;
    float z[kE], x[kE];
    uint32_t w[kE];
    R::unpack(q, z);
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      x_pair(z[e], z[e + 1], m, c, x[e], x[e + 1]);
      weights_of(x[e], x[e + 1], w[e], w[e + 1]);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) sum = add_wide(sum, w[e]);
    if (some) {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (window.has(x[e])) add_to_bin(b, window.at(x[e]), true, w[e]);
    }
  });
  return sum;
}

// The same for counts alone.
template <class B, class R>
__device__ __noinline__ void count(B b, R r, float m, float c, Window window) {
  r.template each<false, 4>([&](int, const uint4& q) {
    if (!(x_of(R::top_of(q), m, c) > -window.to)) return;
    float z[R::kElems];
    R::unpack(q, z);
#pragma unroll
    for (int e = 0; e < R::kElems; ++e) {
      const float x = x_of(z[e], m, c);
      if (window.has(x)) add_to_bin(b, window.at(x), false, 0);
    }
  });
}

// The weight of the thread's elements that are kept: z > cut, or z = cut and id <= cut_id,
// and a weight of `least` or more.
template <class R>
__device__ __noinline__ uint64_t weight_kept(R r, float m, float c, uint32_t least, float cut,
                                             int cut_id) {
  constexpr int kE = R::kElems;
  uint64_t sum = 0;
  r.template each<false, 4>([&](int v, const uint4& q) {
    if (!(R::top_of(q) >= cut)) return;
    float z[kE];
    uint32_t w[kE];
    R::unpack(q, z);
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      float x0, x1;
      x_pair(z[e], z[e + 1], m, c, x0, x1);
      weights_of(x0, x1, w[e], w[e + 1]);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (w[e] >= least && (z[e] > cut || (z[e] == cut && r.id_of(v) + e <= cut_id)))
        sum = add_wide(sum, w[e]);
  });
  return sum;
}

// One warp finds the token among its vectors [v0, v1): the kept weights before them sum to
// `before`, and the running sum of theirs passes `at`.
template <class R>
__device__ __noinline__ void take_token(R r, Filter f, const SampleArgs& a, int row, float cut,
                                        int cut_id, uint64_t before, uint64_t at,
                                        uint64_t total) {
  constexpr int kE = R::kElems;
  const int lane = threadIdx.x & 31;
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
        if (z[e] > cut || (z[e] == cut && r.id_of(v + lane) + e <= cut_id)) {
          w[e] = f.weight(z[e]);
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
        if (prior <= at && at < prior + w[e]) write_answer(a, f, row, r.id_of(v + lane) + e, z[e], total);
        prior += w[e];
      }
    }
    before += __shfl_sync(kFull, upto, 31);
    if (before > at) return;
  }
}

}  // namespace
}  // namespace rlk
