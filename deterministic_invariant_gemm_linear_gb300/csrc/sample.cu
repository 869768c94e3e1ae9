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
// Calls below kStreamBytes run sample_kernel: a cluster of 1 - 16 CTAs takes a row, each CTA a
// contiguous run of its ids.  (Larger calls: see the streaming kernels.)  A row needs one pass
// for its maximum and at least one more, from shared memory (kOnChip) or from L2; what bounds
// the kernel is latency, the chain of passes and cluster barriers: a row of 151,936 FP32
// logits with top-k, top-p and min-p takes 17.8 us, 7 rows of 32,003 in BF16 without any
// 11 us, where their bytes would take 0.1.  No row is sorted:
//  * top-k of few (the usual): a CTA's threads each know their own largest logit, so the
//    k-th largest of those is a value that at least k of the CTA's logits reach.  What
//    reaches it goes to the leading CTA, which sorts those few and finishes the row: one
//    cluster barrier in all.
//  * otherwise: a histogram of x over the 32 octaves that have weight (counts, and weights
//    for top-p), whose bins are runs of the sorted order, gives the bin the cut falls in.
//    If what lies up to that bin is at most kList elements, the leading CTA finishes as
//    above; else it sorts that bin alone to find the cut, and the cluster draws from what
//    lies before it.  A bin of more than kList elements (many equal logits) is narrowed by
//    histograms of the logits' bit patterns to one value, then one id among equal values.
#include <math.h>

#include <mutex>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_pipeline.cuh"
#include "rlk_sample.cuh"

namespace rlk {
namespace {

// Where the kept prefix of the sorted order ends: its last entry (all ones: nowhere), or 0 if
// the leading CTA finished the row from a list.  `top`: the largest of the thread's logits.
template <class B, class R>
__device__ __noinline__ uint64_t search(B b, R r, Filter f, const SampleArgs& a, int row,
                                        float top) {
  constexpr int kE = R::kElems;
  SampleSmem* s = b.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t last = ~0ull;
  bool by_mass = !f.need_k;                        // the search under way
  uint64_t total_mass = 0, want_mass = 0;
  // at most: by count, by weight instead if that cuts nothing, or by weight after it
  for (int pass = 0; pass < 2 && (f.need_k || f.need_p); ++pass) {
    uint32_t before = 0;                           // elements, weight above the range searched
    uint64_t mass_before = 0;
    Cut cut;
    Window window(0.f, f.need_p ? kNear : kOctaves);
    const float top_x = x_of(top, f.m, f.c);       // of this thread's elements
    for (;;) {
      clear_bins(b, f.need_p);
      if (f.need_p) {
        const bool whole = total_mass == 0;        // the row's weight is not known yet
        uint64_t sum = weigh(b, r, f.m, f.c, window, whole);
        if (whole) {
          sum = block_sum(b, sum, 0);
          if (warp == 0) b.push(9, sum);
        }
      } else {
        count(b, r, f.m, f.c, window);
      }
      cluster_join();                              // every CTA's histogram is complete
      if (f.need_p && total_mass == 0) {
        total_mass = b.sum_of(9, b.ctas);
        if (by_mass) want_mass = f.share(total_mass);
      }
      uint32_t all_n;
      uint64_t all_mass;
      cut = find_cut(b, f.need_p, by_mass, f.k - before, want_mass - mass_before, &all_n, &all_mass);
      if (cut.bin >= 0 || window.to >= kOctaves) break;
      before += all_n;
      mass_before += all_mass;
      window = Window(kNear, kOctaves);
    }
    if (cut.bin < 0) {
      // Only weightless elements are left: top-k cuts nothing that could be drawn.
      f.need_k = false;
      if (by_mass || !f.need_p) break;
      by_mass = true;
      want_mass = f.share(total_mass);
      continue;
    }
    before += cut.before;
    mass_before += cut.mass;
    const bool to_end = f.need_k == !by_mass;      // nothing is left to cut after this search
    const bool near = window.bin(top_x) <= cut.bin;
    const float m = f.m, c = f.c;
    const int bin = cut.bin;
    if (tid == 0) s->n_list = 0;
    __syncthreads();
    if (to_end && before + cut.in <= kList) {
      list_range_cold(b, r, near, least_logit(m, c, window, bin), INFINITY);
      push_count(b);
      cluster_join();
      gather_lists(b);
      if (b.rank == 0) finish(b, f, a, row, (int)(before + cut.in), total_mass);
      return 0;
    }
    if (cut.in <= kList) {
      const float lo = least_logit(m, c, window, bin);
      // the bin ends below the least logit of the bins before it
      float hi = m;
      if (bin > 0 || window.from > 0.f) hi = logit_of(key_of(least_logit(m, c, window, bin - 1)) - 1);
      list_range_cold(b, r, near, lo, hi);
      push_count(b);
      cluster_join();
      gather_lists(b);
      if (b.rank == 0) {
        cut_in_bin(b, f, (int)cut.in, by_mass, f.k - before, mass_before, want_mass);
        if (warp == 0) {
          b.push(5, s->total[2]);
          b.push(6, s->total[3]);
        }
      }
      cluster_join();
      last = s->from[5][0];
      mass_before = s->from[6][0];
    } else {
      // ---- too many for a sort: the bin's range of keys, ...
      uint32_t kmin = kFull, kmax = 0;
      r.template each<false, 4>([&](int, const uint4& q) {
        float z[kE];
        R::unpack(q, z);
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (window.bin(x_of(z[e], m, c)) == bin) {
            kmin = min(kmin, key_of(z[e]));
            kmax = max(kmax, key_of(z[e]));
          }
      });
      kmin = __reduce_min_sync(kFull, kmin);
      kmax = __reduce_max_sync(kFull, kmax);
      if (lane == 0) s->part[0][warp] = ((uint64_t)~kmin << 32) | kmax;
      __syncthreads();
      if (warp == 0) {
        const uint64_t v = lane < B::kWarps ? s->part[0][lane] : 0;
        b.push(1, ((uint64_t)__reduce_max_sync(kFull, (uint32_t)(v >> 32)) << 32) |
                      __reduce_max_sync(kFull, (uint32_t)v));
      }
      cluster_join();
      kmin = kmax = 0;
      for (int i = 0; i < b.ctas; ++i) {
        kmin = max(kmin, (uint32_t)(s->from[1][i] >> 32));
        kmax = max(kmax, (uint32_t)s->from[1][i]);
      }
      kmin = ~kmin;
      // ... that range in kBins parts until a part is one key, ...
      uint32_t in = cut.in;
      for (int level = 0; kmin != kmax && level < 4; ++level) {   // 32 bits, 10 a level
        int shift = 0;
        while (((kmax - kmin) >> shift) >= kBins) ++shift;
        clear_bins(b, f.need_p);
        r.template each<false, 4>([&](int, const uint4& q) {
          float z[kE];
          R::unpack(q, z);
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const uint32_t key = key_of(z[e]);
            if (key >= kmin && key <= kmax)
              add_to_bin(b, (kmax - key) >> shift, f.need_p, f.need_p ? f.weight(z[e]) : 0);
          }
        });
        cluster_join();
        uint32_t all_n;
        uint64_t all_mass;
        const Cut part = find_cut(b, f.need_p, by_mass, f.k - before, want_mass - mass_before,
                                  &all_n, &all_mass);
        before += part.before;
        mass_before += part.mass;
        in = part.in;
        const uint32_t hi = kmax - ((uint32_t)part.bin << shift);
        const uint32_t below = (1u << shift) - 1;
        kmin = hi - kmin > below ? hi - below : kmin;
        kmax = hi;
      }
      // ... and how many of the equal ones
      const uint32_t w = f.weight(logit_of(kmax));
      uint64_t keep = in;
      if (!by_mass) keep = f.k - before;
      else if (w) keep = (want_mass - mass_before + w - 1) / w;
      if (keep > in) keep = in;
      mass_before += keep * w;
      uint32_t cut_id = kFull;                     // all of them
      if (keep < in) {
        uint32_t ties = 0;
        r.template each<false, 4>([&](int, const uint4& q) {
          float z[kE];
          R::unpack(q, z);
#pragma unroll
          for (int e = 0; e < kE; ++e) ties += key_of(z[e]) == kmax;
        });
        ties = __reduce_add_sync(kFull, ties);
        const uint64_t here = block_sum(b, lane == 0 ? ties : 0, 0);
        if (warp == 0) b.push(2, here);
        if (tid == 0) s->answer = 0;
        cluster_join();
        uint64_t below = b.sum_of(2, b.rank);      // in earlier CTAs, then in earlier warps
        for (int o = 0; o < warp; ++o) below += s->part[0][o];
        if (below < keep && keep <= below + ties) {   // uniform in the warp: its part has it
          for (int v = r.v0; v < r.v1; v += 32) {
            float z[kE];
            uint32_t n = 0;
            if (v + lane < r.v1) {
              r.get(v + lane, z);
#pragma unroll
              for (int e = 0; e < kE; ++e) n += key_of(z[e]) == kmax;
            }
            uint32_t upto = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const uint32_t o = __shfl_up_sync(kFull, upto, off);
              if (lane >= off) upto += o;
            }
            uint64_t seen = below + upto - n;
            if (seen < keep && keep <= below + upto) {
#pragma unroll
              for (int e = 0; e < kE; ++e)
                if (key_of(z[e]) == kmax && ++seen == keep) s->answer = r.id_of(v + lane) + e;
            }
            below += __shfl_sync(kFull, upto, 31);
          }
        }
        __syncthreads();
        if (warp == 0) b.push(3, (uint64_t)s->answer);
        cluster_join();
        cut_id = (uint32_t)b.max_of(3);
      }
      last = ((uint64_t)~kmax << 32) | cut_id;
    }
    if (by_mass || !f.need_p) break;
    by_mass = true;                                // top-p among the k kept
    want_mass = f.share(mass_before);
  }
  return last;
}

// A row by its cluster.
template <bool kFp32, bool kOnChip, int kT>
__device__ __forceinline__ void sample_row(const Block<kT>& b, const SampleArgs& a, int per,
                                           int row, uint8_t* vectors_at) {
  using R = Row<kFp32, kOnChip>;
  using B = Block<kT>;
  SampleSmem* s = b.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s->n_list = 0;
    s->top = 0;
    s->reached = kFull;
  }
  __syncthreads();
  bool bad;
  Filter f = settings_of(a, row, &bad);
  // ---- the first pass: the largest logit
  R r;
  {
    const int vectors = r.begin(a, row);
    const int cta0 = b.rank * per;
    const int mine = max(0, min(per, vectors - cta0));
    const int each = (mine + B::kWarps - 1) / B::kWarps;
    r.skip(cta0);
    r.chip = reinterpret_cast<uint4*>(vectors_at);
    r.v0 = min(warp * each, mine);
    r.v1 = min(r.v0 + each, mine);
  }
  float top = -INFINITY;
  r.template each<true, 8>([&](int v, const uint4& q) {
    if constexpr (kOnChip) r.chip[v] = q;
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(R::top_of(q)));
  });
  // A key above all logits marks what no token can be drawn from: NaN, +inf, bad settings.
  const uint32_t my_top = bad || !(top < INFINITY) ? kFull : key_of(top);
  const uint32_t warp_top = __reduce_max_sync(kFull, my_top);
  if (lane == 0) atomicMax(&s->top, warp_top);
  __syncthreads();
  const uint32_t cta_top = s->top;
  if (warp == 0) b.push(0, cta_top);

  // ---- top-k of few: what reaches the k-th largest of the threads' own largest
  const bool few = f.need_k && f.k <= kT && f.k * b.ctas <= kList / 2;
  if (few) {
    // Bins below this CTA's largest; what has no weight beside it has none in the row.
    const float m = logit_of(cta_top), c = f.c;
    const int my_bin = cta_top != kFull ? all_octaves().bin(x_of(top, m, c)) : kBins;
    const int reach = reach_bin(my_bin, f.k);
    const uint32_t reached = __reduce_min_sync(kFull, my_bin <= reach ? my_top : kFull);
    if (lane == 0) atomicMin(&s->reached, reached);
    if ((uint32_t)__syncthreads_count(my_bin <= reach) >= f.k) {
      const float least = logit_of(s->reached);
      list_range(b, r, top >= least, least, INFINITY);
    } else if (cta_top != kFull) {                 // fewer have weight than k
      list_range_cold(b, r, my_bin < kBins, least_logit(m, c, all_octaves(), kBins - 1), INFINITY);
    }
    push_count(b);
  }
  cluster_join();
  const uint32_t row_top = (uint32_t)b.max_of(0);
  f.m = logit_of(row_top);
  if (row_top == kFull || f.m == -INFINITY) {      // nothing to draw from
    if (b.rank == 0 && tid == 0 && RLK_STORE_OK(row < a.N, &g_err_sample)) {
      a.token[row] = -1;
      a.logp[row] = __int_as_float(0x7fc00000);
    }
    return;
  }
  if (few) {
    const uint64_t n = b.sum_of(7, b.ctas);
    if (n <= kList) {
      gather_lists(b);
      if (b.rank == 0) finish(b, f, a, row, (int)n, 0);
      return;
    }
  }

  uint64_t last = ~0ull;                           // the last entry kept
  if (f.need_k || f.need_p) {
    last = search(b, r, f, a, row, top);
    if (last == 0) return;
  }

  // ---- the weight kept, by warp and CTA: z > cut, or z = cut and id <= cut_id
  const float cut = last == ~0ull ? -INFINITY : entry_logit(last);
  const int cut_id = last == ~0ull ? -1 : (int)min((uint32_t)last, (uint32_t)a.V);
  uint64_t sum = weight_kept(r, f.m, f.c, f.least, cut, cut_id);
  sum = warp_sum(sum);
  {
    const uint64_t here = block_sum(b, lane == 0 ? sum : 0, 1);
    if (warp == 0) b.push(4, here);
  }
  cluster_join();
  uint64_t before = b.sum_of(4, b.rank);
  const uint64_t total = b.sum_of(4, b.ctas);
  for (int o = 0; o < warp; ++o) before += s->part[1][o];
  const uint64_t at = scaled_31(total, f.u31);
  if (!(before <= at && at < before + sum)) return;   // uniform in the warp: the token is elsewhere
  take_token(r, f, a, row, cut, cut_id, before, at, total);
}

template <bool kFp32, bool kOnChip, int kT>
__global__ void __launch_bounds__(kT, 1024 / kT) sample_kernel(const __grid_constant__ SampleArgs a,
                                                               int per) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Block<kT> b;
  b.s = reinterpret_cast<SampleSmem*>(smem_raw);
  b.rank = (int)cluster_rank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(b.ctas));
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int first = blockIdx.x / b.ctas, clusters = gridDim.x / b.ctas;
  const int rows = a.left ? *a.left : a.N;         // all: a row each
  for (int i = first; i < rows; i += clusters) {
    sample_row<kFp32, kOnChip, kT>(b, a, per, a.left ? a.left[1 + i] : i,
                                   smem_raw + sizeof(SampleSmem));
    if (!a.left) return;
    cluster_join();                                // the shared memory is free again
  }
}

// ---------------------------------------------------------------- streaming kernels
// Calls of many large rows: every pass over the logits is a kernel of independent warps
// without a barrier, which streams, and what belongs to a row as a whole is a CTA's work
// between two passes.  In brackets, us for 512 rows of 152,064 BF16 logits with top-p
// (156 MB) and for 1024 rows of 151,936 FP32 logits (622 MB), five in six greedy or with
// top-k and most of the others with top-p, and what bounds each:
//   tops   the largest logit of every chunk (the 8 vectors a lane of a tile reads)
//          [25, 89; memory: 6.2 and 7.0 TB/s]
//   pick   the row's largest; top-k of at most kChunkTop: the k-th largest of the chunks'
//          bounds the k first, only the chunks that reach it are read again, and the row
//          is done  [10, 54; latency of the lists and their order]
//   weigh  the other rows' weights by tile, for top-p with their histogram
//          [80, 38; instructions: the exact weights alone take 55 of the 80 (the same rows
//          without top-p), the histogram's places and its two shared atomics the rest]
//   cut    rows that keep all: the token's tile by a running sum, then the token; top-p: the
//          bin of the cut from the histogram and, if little lies up to it, the token
//          [24, 21; latency]
//   weigh  again, for the other rows with top-p: the weights above that bin by tile, and its
//          elements in a list  [27, 21; instructions, of the quarter of the rows left]
//   cut    again: the cut from the sorted list, and the token  [25, 20; latency]
// Rows that none of this settles (more equal logits than the list holds, top-k of more, a cut
// in the last octaves) are left to sample_kernel, which takes them from a list.
constexpr int kTile = 256;                    // vectors of a tile: 8 a lane
constexpr int kStreamThreads = 256;           // of the passes
// Of a row's work between them.  More rows at a time hide the short steps that both wait on,
// more threads shorten a row's own: the pick took 62.5 / 230 / 174 us of whole calls (64 and
// 1024 FP32 rows with settings of every kind, 512 BF16 rows with top-p) at 512 threads and 65 /
// 231 / 171 at 256, the cut 62 / 232 / 197 at 512 and 63 / 233 / 181 at 256 (when each was set).
constexpr int kPickThreads = 512, kCutThreads = 256;
// Tiles a CTA of the weighing kernels: the most, and half of them in calls that have at most
// kFewCtas CTAs an SM with the most (us of whole calls, half against the most: with top-p 64 rows
// of FP32 64 / 69, 128 of BF16 82 / 90, 256 of BF16 119 / 126, 384 of FP32 171 / 168; settings of
// every kind, FP32, 64 rows 60 / 65, 1024 rows 238 / 229).
constexpr int kTilesPerCta = 16;
constexpr int kFewCtas = 13;
constexpr int kChunkTop = 1024;

// What the streaming kernels know of a row between them.
enum RowStatus { kDone = 0, kWeigh = 1, kWeighBins = 2, kCutBin = 3, kLeft = 4 };
struct RowState {
  int status;
  float m;                  // its largest logit
  float lo, hi;             // kCutBin: the logits of the bin the cut falls in
  uint64_t mass_before;     // the weight above the bin, and the weight wanted
  uint64_t mass_wanted;
  int listed;               // the bin's elements listed so far
};

struct StreamArgs {
  SampleArgs a;
  int tiles;                // per row
  int per_cta;              // of the weighing kernels, kTilesPerCta at most
  uint32_t* tops;           // [N][tiles * 32] keys
  uint64_t* mass;           // [N][tiles]
  uint64_t* bin_mass;       // [N][kBins]
  RowState* state;          // [N]
  uint64_t* list;           // [N][kList] the elements of the bins the cuts fall in
  int* left;                // number of rows left to sample_kernel, then the rows
};

__device__ __forceinline__ void put_state(const StreamArgs& p, int row, const RowState& st) {
  if (!RLK_STORE_OK(row < p.a.N, &g_err_sample)) return;
  p.state[row] = st;
  if (st.status == kLeft) {
    const int at = atomicAdd(p.left, 1);           // in any order
    if (RLK_STORE_OK(at < p.a.N, &g_err_sample)) p.left[1 + at] = row;
  }
}

__device__ __forceinline__ void stream_begin() {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
}

// The warp's vectors of tile t.
template <class R>
__device__ __forceinline__ void at_tile(R& r, int vectors, int t) {
  r.v0 = t * kTile;
  r.v1 = min(r.v0 + kTile, vectors);
}

template <bool kFp32>
__global__ void __launch_bounds__(kStreamThreads) sample_tops_kernel(const __grid_constant__ StreamArgs p,
                                                                    int per_row) {
  using R = Row<kFp32, false>;
  stream_begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.left = 0;
  const int row = blockIdx.x / per_row, lane = threadIdx.x & 31;
  const int t = (blockIdx.x - row * per_row) * (kStreamThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.tiles) return;
  R r;
  at_tile(r, r.begin(p.a, row), t);
  float top = -INFINITY;
  r.template each<true, 8>([&](int, const uint4& q) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(R::top_of(q)));
  });
  if (RLK_STORE_OK(row < p.a.N && t < p.tiles, &g_err_sample))
    p.tops[((int64_t)row * p.tiles + t) * 32 + lane] = top < INFINITY ? key_of(top) : kFull;
}

// A CTA's own histogram as scan_cut takes it.
template <class B>
__device__ __forceinline__ void merge_own(const B& b, bool mass) {
  SampleSmem* s = b.s;
  for (int i = threadIdx.x; i < kBins; i += B::kThreads) {
    s->slice_count[i] = s->count[i];
    if (mass) s->slice_mass[i] = s->lo[i] + ((uint64_t)s->hi[i] << 16);
  }
  __syncthreads();
}

// Vectors with an element for the list.
constexpr int kHits = 512;
struct alignas(16) Hits {
  uint4 q[kHits];
  int id[kHits];            // of the vector's first element
  uint32_t n;               // kHits and more of them are taken one by one
};

template <class R>
__device__ __noinline__ void list_vector(SampleSmem* s, uint4 q, int id, float lo) {
  float z[R::kElems];
  R::unpack(q, z);
#pragma unroll
  for (int e = 0; e < R::kElems; ++e)
    if (z[e] >= lo) {
      const uint32_t to = atomicAdd(&s->n_list, 1u);
      if (to < kList) s->list[to] = entry_of(z[e], id + e);
    }
}

// The chunks whose largest reaches lo, then their elements that do, into the list: the number
// of elements (more than kList: only counted).  ids: [tiles * 32] in shared memory.  The
// vectors with such elements are gathered first and dealt out an element a thread: taken by
// the thread that read them, eight unrolled vectors were 5 us of code run once.
template <class B, class R>
__device__ __noinline__ int list_chunks(B b, R r, int vectors, const uint32_t* tops, int chunks,
                                        float lo, uint16_t* ids, Hits* hits) {
  constexpr int kE = R::kElems;
  SampleSmem* s = b.s;
  const uint32_t least = key_of(lo);
  __syncthreads();
  if (threadIdx.x == 0) {
    s->n_list = 0;
    s->n_chunks = 0;
    hits->n = 0;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < chunks; i0 += 8 * B::kThreads) {
    uint32_t key[8], mine = 0;                     // all eight loads before the first use
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * B::kThreads + threadIdx.x;
      key[j] = i < chunks ? tops[i] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += key[j] >= least && key[j];
    uint32_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(kFull, upto, off);
      if (lane >= off) upto += o;
    }
    uint32_t at = 0;
    if (lane == 31 && upto) at = atomicAdd(&s->n_chunks, upto);
    at = __shfl_sync(kFull, at, 31) + upto - mine;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (key[j] >= least && key[j]) ids[at++] = (uint16_t)(i0 + j * B::kThreads + threadIdx.x);
  }
  __syncthreads();
  r.v0 = 0;
  r.v1 = vectors;
  const int n = (int)s->n_chunks;
  for (int i0 = 0; i0 < n; i0 += B::kThreads) {
    const int i = i0 + threadIdx.x;
    if (i < n) {
      const int chunk = ids[i];
      int v[8];
      uint4 q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = min((chunk >> 5) * kTile + 32 * j + (chunk & 31), vectors);
      r.template get_all<true>(v, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (v[j] >= vectors || !(R::top_of(q[j]) >= lo)) continue;
        const uint32_t to = atomicAdd(&hits->n, 1u);
        if (to < kHits) {
          hits->q[to] = q[j];
          hits->id[to] = r.id_of(v[j]);
        } else {
          list_vector<R>(s, q[j], r.id_of(v[j]), lo);
        }
      }
    }
    __syncthreads();
    const int elements = kE * (int)min(hits->n, (uint32_t)kHits);
    for (int t = threadIdx.x; t < elements; t += B::kThreads) {
      const float z = R::element(hits->q, t);
      if (z >= lo) {
        const uint32_t to = atomicAdd(&s->n_list, 1u);
        if (to < kList) s->list[to] = entry_of(z, hits->id[t / kE] + t % kE);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) hits->n = 0;
    if (i0 + B::kThreads < n) __syncthreads();
  }
  return (int)s->n_list;
}

template <bool kFp32>
__global__ void __launch_bounds__(kPickThreads, 2) sample_pick_kernel(const __grid_constant__ StreamArgs p) {
  using R = Row<kFp32, false>;
  using B = Block<kPickThreads>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  B b;
  b.s = reinterpret_cast<SampleSmem*>(smem_raw);
  b.rank = 0;
  b.ctas = 1;
  SampleSmem* s = b.s;
  const int chunks = p.tiles * 32;
  Hits* hits = reinterpret_cast<Hits*>(smem_raw + sizeof(SampleSmem));
  uint32_t* tops = reinterpret_cast<uint32_t*>(hits + 1);
  uint16_t* ids = reinterpret_cast<uint16_t*>(tops + chunks);
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) s->top = 0;
  clear_bins(b, false);
  stream_begin();
  bool bad;
  Filter f = settings_of(p.a, row, &bad);
  const uint32_t* src = p.tops + (int64_t)row * chunks;
  uint32_t top = 0;
#pragma unroll 8
  for (int i = tid; i < chunks; i += kPickThreads) {
    const uint32_t key = __ldg(src + i);
    tops[i] = key;
    top = max(top, key);
  }
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) atomicMax(&s->top, top);
  __syncthreads();
  top = s->top;
  f.m = logit_of(top);
  RowState st;
  st.status = kDone;
  st.m = f.m;
  st.lo = st.hi = 0.f;
  st.mass_before = st.mass_wanted = 0;
  st.listed = 0;
  if (bad || top == kFull || f.m == -INFINITY) {
    if (tid == 0 && RLK_STORE_OK(row < p.a.N, &g_err_sample)) {
      p.a.token[row] = -1;
      p.a.logp[row] = __int_as_float(0x7fc00000);
    }
  } else if (f.need_k) {
    st.status = kLeft;
    if (f.k <= kChunkTop && (int)f.k <= chunks / 2) {
      for (int i = tid; i < chunks; i += kPickThreads) {
        const int bin = all_octaves().bin(x_of(logit_of(tops[i]), f.m, f.c));
        if (bin < kBins) add_to_bin(b, bin, false, 0);
      }
      uint32_t all_n;
      uint64_t all_mass;
      if (tid == 0) s->cut.bin = -1;
      __syncthreads();
      merge_own(b, false);
      const Cut cut = scan_cut(b, false, false, f.k, 0, &all_n, &all_mass);
      // fewer chunks have weight than k: all that has weight
      const float lo = least_logit(f.m, f.c, all_octaves(), cut.bin >= 0 ? cut.bin : kBins - 1);
      R r;
      const int vectors = r.begin(p.a, row);
      const int n = list_chunks(b, r, vectors, tops, chunks, lo, ids, hits);
      if (n <= kList) {
        finish(b, f, p.a, row, n, 0);
        st.status = kDone;
      }
    }
  } else {
    st.status = f.need_p ? kWeighBins : kWeigh;
    if (f.need_p)
      for (int i = tid; i < kBins; i += kPickThreads)
        if (RLK_STORE_OK(row < p.a.N, &g_err_sample)) p.bin_mass[(int64_t)row * kBins + i] = 0;
  }
  if (tid == 0) put_state(p, row, st);
}

// A tile CTA's histogram holds weights as two halves whose sums fit 32 bits: it has at most
// 2^15 elements.  Most weights of an open row have no high part (14 octaves below the top).
// Shared atomics on scattered bins are what the pass waits for, so elements are not counted:
// a bin's weights are alike, and its weight bounds their number.
constexpr int kLowBits = 17;
constexpr uint32_t kLowPart = (1u << kLowBits) - 1;
static_assert(kTilesPerCta * kTile * 8 <= 1 << (32 - kLowBits), "sums of low parts fit 32 bits");

// At most so many elements make up the weight of a bin of the first octaves: each lies at
// most bin + 1/2 steps below the top (2^(1/2 step) is room for rounding).
__device__ __forceinline__ uint32_t most_in(const Window& window, int bin, uint64_t mass) {
  return (uint32_t)__fmul_rn(__ull2float_rn(mass), exp2f((bin + 1) / window.scale - 31.f));
}

// The elements of the cut's bin that a CTA found, at most all of them.  They join the row's
// list by one addition to its length: one addition an element, each waited for, made the pass
// 31 us instead of 28 (512 rows of BF16, a quarter of them still under way).
struct Found {
  uint64_t entry[kList];
  uint32_t n, at;
};

// The weight of tiles: of the rows that keep all (but what min-p drops) and, with their
// histogram over the first octaves, of the rows with top-p; or (kAbove) of what lies above
// the bin the cut falls in, with a list of the bin's elements.
enum WeighWhat { kAll, kAtLeast, kBinned, kAboveBin };
template <bool kFp32, WeighWhat kWhat>
__device__ __forceinline__ void weigh_tiles(const StreamArgs& p, int row, int t0, int t1,
                                            const RowState& st, float c, uint32_t least,
                                            uint32_t* lo, uint32_t* hi, Found* found) {
  using R = Row<kFp32, false>;
  constexpr int kE = R::kElems;
  const Window window(0.f, kNear);
  R r;
  const int vectors = r.begin(p.a, row);
  for (int t = t0 + (threadIdx.x >> 5); t < t1; t += kStreamThreads / 32) {
    at_tile(r, vectors, t);
    uint64_t sum = 0;
    r.template each<true, 4>([&](int v, const uint4& q) {
      if (kWhat == kAboveBin && !(R::top_of(q) >= st.lo)) return;
      float z[kE], x[kE];
      uint32_t w[kE];
      R::unpack(q, z);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        x_pair(z[e], z[e + 1], st.m, c, x[e], x[e + 1]);
        weights_of(x[e], x[e + 1], w[e], w[e + 1]);
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        bool keep = true;
        if (kWhat == kAtLeast) keep = w[e] >= least;
        if (kWhat == kAboveBin) {
          keep = z[e] > st.hi && w[e] >= least;
          if (z[e] >= st.lo && z[e] <= st.hi) {
            const uint32_t at = atomicAdd(&found->n, 1u);        // in any order: it is sorted
            if (at < kList) found->entry[at] = entry_of(z[e], r.id_of(v) + e);
          }
        }
        if (keep) sum = add_wide(sum, w[e]);
      }
      if (kWhat == kBinned && x_of(R::top_of(q), st.m, c) > -window.to) {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (x[e] > -window.to) {               // and none lies above the top
            const int bin = window.at(x[e]);
            atomicAdd(&lo[bin], w[e] & kLowPart);
            atomicAdd(&hi[bin], w[e] >> kLowBits);
          }
      }
    });
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0 && RLK_STORE_OK(row < p.a.N && t < p.tiles, &g_err_sample))
      p.mass[(int64_t)row * p.tiles + t] = sum;
  }
}

template <bool kFp32, bool kAbove>
__global__ void __launch_bounds__(kStreamThreads) sample_weigh_kernel(const __grid_constant__ StreamArgs p,
                                                                     int per_row) {
  __shared__ uint32_t lo[kAbove ? 1 : kBins], hi[kAbove ? 1 : kBins];
  stream_begin();
  const int row = blockIdx.x / per_row;
  const RowState st = p.state[row];
  if (kAbove ? st.status != kCutBin : st.status != kWeigh && st.status != kWeighBins) return;
  const int t0 = (blockIdx.x - row * per_row) * p.per_cta, t1 = min(t0 + p.per_cta, p.tiles);
  bool bad;
  const Filter f = settings_of(p.a, row, &bad);
  if (kAbove) {
    __shared__ Found found;
    if (threadIdx.x == 0) found.n = 0;
    __syncthreads();
    weigh_tiles<kFp32, kAboveBin>(p, row, t0, t1, st, f.c, f.least, lo, hi, &found);
    __syncthreads();
    const int n = (int)min(found.n, (uint32_t)kList);
    if (n == 0) return;
    if (threadIdx.x == 0) found.at = (uint32_t)atomicAdd(&p.state[row].listed, n);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kStreamThreads)
      if (found.at + i < kList && RLK_STORE_OK(row < p.a.N, &g_err_sample))
        p.list[(int64_t)row * kList + found.at + i] = found.entry[i];
  } else if (st.status == kWeigh) {
    if (f.least == 0)
      weigh_tiles<kFp32, kAll>(p, row, t0, t1, st, f.c, 0, lo, hi, nullptr);
    else
      weigh_tiles<kFp32, kAtLeast>(p, row, t0, t1, st, f.c, f.least, lo, hi, nullptr);
  } else {
    for (int i = threadIdx.x; i < kBins; i += kStreamThreads) lo[i] = hi[i] = 0;
    __syncthreads();
    weigh_tiles<kFp32, kBinned>(p, row, t0, t1, st, f.c, 0, lo, hi, nullptr);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kStreamThreads)
      if ((lo[i] | hi[i]) && RLK_STORE_OK(row < p.a.N, &g_err_sample))
        // sums of whole numbers: their order does not matter
        atomicAdd(reinterpret_cast<unsigned long long*>(&p.bin_mass[(int64_t)row * kBins + i]),
                  (unsigned long long)lo[i] + ((unsigned long long)hi[i] << kLowBits));
  }
}

// The token of a row whose tiles' kept weights are known: its tile, then itself.
template <class B, class R>
__device__ __forceinline__ void draw(const B& b, const StreamArgs& p, int row, const Filter& f, R r,
                                     int vectors, float cut, int cut_id) {
  SampleSmem* s = b.s;
  const uint64_t* mass = p.mass + (int64_t)row * p.tiles;
  const int each = (p.tiles + B::kThreads - 1) / B::kThreads;
  const int t0 = min((int)threadIdx.x * each, p.tiles), t1 = min(t0 + each, p.tiles);
  uint64_t sum = 0;
  for (int t = t0; t < t1; ++t) sum += __ldcg(mass + t);   // some just added to
  uint64_t upto = sum;
  uint32_t unused = 0;
  block_scan(b, unused, upto);
  if (threadIdx.x == B::kThreads - 1) s->total[0] = upto;
  __syncthreads();
  const uint64_t total = s->total[0];
  const uint64_t at = scaled_31(total, f.u31);
  uint64_t before = upto - sum;
  if (before <= at && at < upto)                   // one thread's tiles
    for (int t = t0; t < t1; ++t) {
      const uint64_t here = __ldcg(mass + t);
      if (at < before + here) {
        s->answer = t;
        s->total[1] = before;
        break;
      }
      before += here;
    }
  __syncthreads();
  if (threadIdx.x < 32) {
    at_tile(r, vectors, s->answer);
    take_token(r, f, p.a, row, cut, cut_id, s->total[1], at, total);
  }
}

template <bool kFp32>
__global__ void __launch_bounds__(kCutThreads, 1024 / kCutThreads)
    sample_cut_kernel(const __grid_constant__ StreamArgs p, int again) {
  using R = Row<kFp32, false>;
  using B = Block<kCutThreads>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  B b;
  b.s = reinterpret_cast<SampleSmem*>(smem_raw);
  b.rank = 0;
  b.ctas = 1;
  SampleSmem* s = b.s;
  Hits* hits = reinterpret_cast<Hits*>(smem_raw + sizeof(SampleSmem));
  uint16_t* ids = reinterpret_cast<uint16_t*>(hits + 1);
  const int row = blockIdx.x, tid = threadIdx.x;
  stream_begin();
  RowState st = p.state[row];
  if (again ? st.status != kCutBin : st.status != kWeigh && st.status != kWeighBins) return;
  bool bad;
  Filter f = settings_of(p.a, row, &bad);
  f.m = st.m;
  R r;
  const int vectors = r.begin(p.a, row);
  float cut = -INFINITY;                           // kept: z > cut, or z = cut and id <= cut_id
  int cut_id = -1;
  if (st.status == kCutBin) {
    const int n = min(st.listed, kList);           // no more than the histogram's weight bounds
    const uint64_t* list = p.list + (int64_t)row * kList;
    // the part of the bin that the cut falls in, and its elements alone sorted
    const uint32_t high = key_of(st.hi), range = high - key_of(st.lo);
    const int shift = range < kBins ? 0 : 32 - __clz((int)(range / kBins));
    clear_bins(b, true);
    for (int i = tid; i < n; i += kCutThreads) {
      const uint64_t x = __ldg(list + i);
      add_to_bin(b, (int)((high - ~(uint32_t)(x >> 32)) >> shift), true, f.weight(entry_logit(x)));
    }
    if (tid == 0) {
      s->cut.bin = -1;
      s->n_list = 0;
    }
    __syncthreads();
    merge_own(b, true);
    uint32_t all_n;
    uint64_t all_mass;
    const Cut part = scan_cut(b, true, true, 0, st.mass_wanted - st.mass_before, &all_n, &all_mass);
    for (int i = tid; i < n; i += kCutThreads) {
      const uint64_t x = __ldg(list + i);
      if ((int)((high - ~(uint32_t)(x >> 32)) >> shift) == part.bin)
        s->list[atomicAdd(&s->n_list, 1u)] = x;
    }
    __syncthreads();
    cut_in_bin(b, f, (int)part.in, true, 0, st.mass_before + part.mass, st.mass_wanted);
    const uint64_t last = s->total[2];
    cut = entry_logit(last);
    cut_id = (int)(uint32_t)last;
    // the bin's kept elements join their tiles
    for (int i = tid; i < n; i += kCutThreads) {
      const uint64_t x = __ldg(list + i);
      const uint32_t w = f.weight(entry_logit(x));
      const int t = ((int)(uint32_t)x - r.first_id) / R::kElems / kTile;
      if (x <= last && w >= f.least && RLK_STORE_OK(row < p.a.N && t < p.tiles, &g_err_sample))
        atomicAdd(reinterpret_cast<unsigned long long*>(&p.mass[(int64_t)row * p.tiles + t]),
                  (unsigned long long)w);
    }
    __syncthreads();
  }
  if (st.status != kWeighBins) {
    draw(b, p, row, f, r, vectors, cut, cut_id);
    return;
  }
  const int chunks = p.tiles * 32;
  const uint32_t* tops = p.tops + (int64_t)row * chunks;
  // the row's weight, its histogram, the cut's bin
  uint64_t sum = 0;
  for (int t = tid; t < p.tiles; t += kCutThreads) sum += p.mass[(int64_t)row * p.tiles + t];
  sum = block_sum(b, sum, 0);
  if (tid == 0) {
    s->total[2] = sum;
    s->cut.bin = -1;
  }
  const Window window(0.f, kNear);
  for (int i = tid; i < kBins; i += kCutThreads) {
    const uint64_t in = p.bin_mass[(int64_t)row * kBins + i];
    s->slice_count[i] = most_in(window, i, in);
    s->slice_mass[i] = in;
  }
  __syncthreads();
  const uint64_t total = s->total[2], want = f.share(total);
  uint32_t all_n;
  uint64_t all_mass;
  const Cut found = scan_cut(b, true, true, 0, want, &all_n, &all_mass);
  st.status = kLeft;
  if (found.bin >= 0 && found.before + found.in <= kCutThreads) {
    const float lo = least_logit(f.m, f.c, window, found.bin);
    const int n = list_chunks(b, r, vectors, tops, chunks, lo, ids, hits);
    finish(b, f, p.a, row, n, total);
    st.status = kDone;
  } else if (found.bin >= 0 && found.in <= kList) {
    st.lo = least_logit(f.m, f.c, window, found.bin);
    st.hi = f.m;
    if (found.bin > 0) st.hi = logit_of(key_of(least_logit(f.m, f.c, window, found.bin - 1)) - 1);
    st.mass_before = found.mass;
    st.mass_wanted = want;
    st.status = kCutBin;
  }
  if (tid == 0) put_state(p, row, st);
}

std::mutex g_attr_mutex;
bool g_attr_set[64];

cudaError_t ensure_attrs(int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_attr_set[dev]) return cudaSuccess;
  cudaError_t e = cudaSuccess;
  for (auto* kernel : {sample_kernel<false, false, 256>, sample_kernel<false, true, 512>,
                       sample_kernel<true, false, 256>, sample_kernel<true, true, 512>}) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  }
  for (auto* kernel : {sample_pick_kernel<false>, sample_pick_kernel<true>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  for (auto* kernel : {sample_cut_kernel<false>, sample_cut_kernel<true>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e == cudaSuccess) g_attr_set[dev] = true;
  return e;
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Logits from which the streaming kernels run, for rows of kStreamVocab or more.  The size alone
// decides, so that it decides the workspace too; the settings do not agree where to change over.
// us of calls over rows of 151,936 FP32 logits, streaming against clusters, with settings for the
// call (top-k and top-p / top-p / neither) and of every kind:
//    8 rows  34 / 44 / 40 / 55   against  26 /  56 / 26 /  33     (4.6 MiB)
//   12 rows  34 / 45 / 40 / 53   against  26 /  77 / 34 /  51
//   16 rows  32 / 46 / 40 / 55   against  29 /  79 / 38 /  53     (9.3 MiB)
//   24 rows  33 / 49 / 39 / 53   against  31 / 126 / 63 /  79
//   48 rows  33 / 62 / 38 / 58   against  42 / 149 / 73 / 112
// so at the change-over top-k loses 10% where top-p gains 40%.  In captured graphs, whose launches
// cost less, 8 rows take 15 / 42 / 17 / 23 against 23 / 56 / 23 / 32.  1024 rows of BF16 (8 MiB
// from 4096 ids on), by vocabulary:
//   12,000   41 /  86 / 43 / 117  against  38 /  97 /  53 /  79
//   16,000   44 /  91 / 48 / 126  against  41 / 136 /  61 / 114
//   24,000   47 / 110 / 57 / 135  against  52 / 167 /  86 / 109
//   32,000   50 / 122 / 64 / 105  against  57 / 187 / 103 / 131
constexpr int64_t kStreamBytes = int64_t(8) << 20;
constexpr int64_t kStreamVocab = 16384;

// How a call runs: the streaming kernels, or clusters of CTAs that keep a row in shared
// memory or read it again from L2.
struct SamplePlan {
  bool stream;
  int ctas;
  bool on_chip;
  int tiles;
  size_t off_mass, off_bins, off_state, off_left, off_list, total;   // their workspace
};

SamplePlan sample_plan(int64_t N, int64_t V, bool fp32, int sms) {
  SamplePlan p = {};
  const int esize = fp32 ? 4 : 2, elems = 16 / esize;
  p.stream = V >= kStreamVocab && N * V * esize >= kStreamBytes;
  if (p.stream) {
    p.tiles = (int)ceil_div(ceil_div(V + elems - 1, elems), kTile);
    p.off_mass = align_up((size_t)N * p.tiles * 32 * sizeof(uint32_t), 256);
    p.off_bins = align_up(p.off_mass + (size_t)N * p.tiles * sizeof(uint64_t), 256);
    p.off_state = align_up(p.off_bins + (size_t)N * kBins * sizeof(uint64_t), 256);
    p.off_left = align_up(p.off_state + (size_t)N * sizeof(RowState), 256);
    p.off_list = align_up(p.off_left + (size_t)(N + 1) * sizeof(int), 256);
    p.total = align_up(p.off_list + (size_t)N * kList * sizeof(uint64_t), 256);
    p.ctas = 1;
    while (p.ctas < kMaxCluster && ceil_div(V, p.ctas) > 60000) p.ctas *= 2;
    return p;
  }
  p.ctas = 1;
  // a CTA has fewer than 2^16 elements (its histogram's halves are 32-bit sums)
  while (p.ctas < kMaxCluster && ceil_div(V, p.ctas) > 60000) p.ctas *= 2;
  while (p.ctas < kMaxCluster && N * p.ctas * 2 <= sms && V / (2 * p.ctas) >= 2048) p.ctas *= 2;
  p.on_chip = N * p.ctas <= 2 * sms && ceil_div(V, p.ctas) * esize <= 77824;
  return p;
}

// The clusters' kernel over all rows, or (left) the rows of that list.
cudaError_t launch_clusters(SampleArgs a, bool fp32, const SamplePlan& plan, const int* left,
                            int sms, cudaStream_t stream) {
  const int elems = fp32 ? 4 : 8;
  a.left = left;
  int64_t clusters = a.N;
  if (left && clusters * plan.ctas > 4 * sms) clusters = 4 * sms / plan.ctas;
  // vectors of a row that starts anywhere in its first vector, dealt evenly
  const int per = (int)ceil_div(ceil_div((int64_t)a.V + elems - 1, elems), plan.ctas);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * plan.ctas));
  cfg.blockDim = dim3(plan.on_chip ? 512 : 256);
  cfg.dynamicSmemBytes = sizeof(SampleSmem) + (plan.on_chip ? (size_t)per * 16 : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)plan.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return fp32 ? (plan.on_chip ? cudaLaunchKernelEx(&cfg, sample_kernel<true, true, 512>, a, per)
                              : cudaLaunchKernelEx(&cfg, sample_kernel<true, false, 256>, a, per))
              : (plan.on_chip ? cudaLaunchKernelEx(&cfg, sample_kernel<false, true, 512>, a, per)
                              : cudaLaunchKernelEx(&cfg, sample_kernel<false, false, 256>, a, per));
}

template <bool kFp32>
cudaError_t launch_stream(const SampleArgs& a, const SamplePlan& plan, uint8_t* ws, int sms,
                          cudaStream_t stream) {
  StreamArgs p;
  p.a = a;
  p.tiles = plan.tiles;
  p.tops = reinterpret_cast<uint32_t*>(ws);
  p.mass = reinterpret_cast<uint64_t*>(ws + plan.off_mass);
  p.bin_mass = reinterpret_cast<uint64_t*>(ws + plan.off_bins);
  p.state = reinterpret_cast<RowState*>(ws + plan.off_state);
  p.left = reinterpret_cast<int*>(ws + plan.off_left);
  p.list = reinterpret_cast<uint64_t*>(ws + plan.off_list);
  const int top_ctas = (int)ceil_div(plan.tiles, kStreamThreads / 32);
  const bool few = a.N * ceil_div(plan.tiles, kTilesPerCta) <= kFewCtas * sms;
  p.per_cta = few ? kTilesPerCta / 2 : kTilesPerCta;
  const int weigh_ctas = (int)ceil_div(plan.tiles, p.per_cta);
  const size_t smem_ids = sizeof(SampleSmem) + sizeof(Hits) + (size_t)plan.tiles * 32 * sizeof(uint16_t);
  const size_t smem_pick = smem_ids + (size_t)plan.tiles * 32 * sizeof(uint32_t);
  const dim3 rows((unsigned)a.N), tops((unsigned)(a.N * top_ctas)), weighs((unsigned)(a.N * weigh_ctas));
  // Passes that settings shared by all rows leave nothing to do for are not launched.
  const bool all_greedy = !a.temperature && a.temperature_all < 1e-6f;
  const bool all_few = all_greedy || (!a.top_k && a.top_k_all > 0 && a.top_k_all <= kChunkTop &&
                                      a.top_k_all <= plan.tiles * 16 && a.top_k_all < a.V);
  const bool any_top_p = !all_few && (a.top_p || a.top_p_all < 1.f);
  cudaError_t e = launch_overlapped(sample_tops_kernel<kFp32>, tops, kStreamThreads, 0, stream, p,
                                    top_ctas);
  if (e == cudaSuccess)
    e = launch_overlapped(sample_pick_kernel<kFp32>, rows, kPickThreads, smem_pick, stream, p);
  for (int again = 0; again < (all_few ? 0 : any_top_p ? 2 : 1) && e == cudaSuccess; ++again) {
    e = again ? launch_overlapped(sample_weigh_kernel<kFp32, true>, weighs, kStreamThreads, 0,
                                  stream, p, weigh_ctas)
              : launch_overlapped(sample_weigh_kernel<kFp32, false>, weighs, kStreamThreads, 0,
                                  stream, p, weigh_ctas);
    if (e == cudaSuccess)
      e = launch_overlapped(sample_cut_kernel<kFp32>, rows, kCutThreads, smem_ids, stream, p, again);
  }
  if (e != cudaSuccess) return e;
  return launch_clusters(a, kFp32, plan, p.left, sms, stream);
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

extern "C" {

size_t rlk_sample_logits_workspace_size(int logits_dtype, int64_t N, int64_t V) {
  if (N < 0 || N >= kMaxSampleRows || V < 1 || V > kMaxSampleVocab ||
      (logits_dtype != RLK_BF16 && logits_dtype != RLK_FP32))
    return 0;
  return sample_plan(N, V, logits_dtype == RLK_FP32, 0).total;
}

rlk_status rlk_sample_logits(const void* logits, int logits_dtype, int64_t N, int64_t V,
                                        int64_t ld, const void* uniform, int uniform_dtype,
                                        const float* temperature, float temperature_all,
                                        const int32_t* top_k, int32_t top_k_all,
                                        const float* top_p, float top_p_all, const float* min_p,
                                        float min_p_all, int64_t* token, float* logp,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  RLK_CALL_RANGE();
  if (N < 0 || N >= kMaxSampleRows || V < 1 || V > kMaxSampleVocab || ld < V ||
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
  const size_t need = rlk_sample_logits_workspace_size(logits_dtype, N, V);
  if (need > 0 && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < need))
    return RLK_ERR_WORKSPACE;
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
  a.fp32 = fp32;
  a.token = token;
  a.logp = logp;
  a.left = nullptr;
  const SamplePlan plan = sample_plan(N, V, fp32, dev.sm_count);
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaError_t e = !plan.stream ? launch_clusters(a, fp32, plan, nullptr, dev.sm_count, q)
                        : fp32       ? launch_stream<true>(a, plan, ws, dev.sm_count, q)
                                     : launch_stream<false>(a, plan, ws, dev.sm_count, q);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return RLK_OK;
}

}  // extern "C"
