// Embedding lookup and its gradient on sm_103a.
//
//   out[r, :] = s W[id_r, :]           dW[v, :] = s sum_{r: id_r = v} d[r, :]
//
// Both are bound by HBM.  The lookup reads N rows and writes N rows.  The gradient writes the
// whole table (V H elements, most of the bytes) and reads the N rows of d once.
//
// The gradient's order is fixed without atomics on numbers: the rows are sorted by id, rows of
// one id in ascending order, and each table row adds its own rows in that order (groups of 64,
// then the groups' sums), so its bits depend on its own rows of d alone.
//  * embed_sort_kernel: the whole sort in one launch, with no exchange between CTAs.  CTA j owns
//    1024 ids and reads all N ids: how many are smaller says where its part of the order begins;
//    its warps, each over its own stretch of the rows, count its ids and then place their rows
//    (equal ids of a warp's 32 rows are ranked by match_any).  N ids are read by V / 1024 CTAs
//    from L2, which for N rows of H elements of d is less than reading d.
//    Its cost, and that of looking through the offsets below, goes with V however few rows there
//    are: one row added to 151936 x 4096 takes 60 us, 64 rows 65, 16384 rows 185.
//  * embed_rows_kernel: every table row.  Most are zeros; an id of at most 64 rows is summed by the
//    threads of its table row.  Ids with more (a padding or a common token can have most of the
//    rows) are cut into groups of 64 for the launch's first blocks; the block that finds all of
//    an id's groups summed (a count says so, the sums lie in the workspace) adds them, in their
//    order, and writes the table row.  No block waits for another.  Those sums are added one after
//    another: 2^20 rows of 256 columns, half of them one id, take 1.84 ms, without that id 0.58.
#include <math.h>

#include <mutex>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_rows.cuh"

namespace rlk {

__device__ unsigned int g_err_embedding = 0;

namespace {

// ---------------------------------------------------------------- lookup
// A row to the threads of row_lanes, each thread's loads of a row before its stores.  16384 x 5120
// BF16: 41 us, 335 MB moved of which common rows come from L2; one row 3.5 us, all of it latency.
template <bool kWFp32, bool kOutFp32, int kRun>
__global__ void __launch_bounds__(kRowThreads)
    embed_kernel(const int64_t* __restrict__ ids, int64_t ids_stride, int64_t N,
                 const void* __restrict__ weight, int64_t V, int H, int64_t ldw, float scale,
                 void* __restrict__ out, int64_t ldo, RowLanes<kRun> lanes) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int64_t r = (int64_t)blockIdx.x * lanes.rows() + lanes.row();
  if (r >= N) return;
  const int64_t id = __ldg(ids + r * ids_stride);
  const bool known = id >= 0 && id < V;
  const int gap = lanes.gap();
  for (int c = lanes.col(); c < H; c += lanes.step()) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (known) {
      load8<kWFp32, kRun>(weight, id * ldw, c, gap, H, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], scale);
    }
    if (RLK_STORE_OK(r < N && min(c + run_at<kRun>(7, gap) + 1, H) <= ldo, &g_err_embedding))
      store8<kOutFp32, kRun>(out, r * ldo, c, gap, H, v);
  }
}

// ---------------------------------------------------------------- gradient: the sort
constexpr int kSortIds = 1024;        // ids a CTA owns, one a thread
constexpr int kSortWarps = kSortIds / 32;
constexpr int kSortCounts = kSortWarps * kSortIds * 4;  // bytes: a count for each warp and id
// rows whose id - lo (kNoKey: another CTA's) waits in shared memory
constexpr int kSortKeys = 32768;
constexpr uint16_t kNoKey = 0xffff;
inline int sort_smem(int64_t N) {
  return kSortCounts + (N <= kSortKeys ? 2 * (int)align_up(N, 32) : 0);
}
constexpr int kGroup = RLK_EMBED_GROUP;

// First group of an id with more than kGroup rows, from the place of its first row: c rows make
// ceil(c / 64) <= 2 c / 65 groups for every c > 64, so no two ids share one, N rows have at most
// 2 N / 65, and nobody has to count them.
__host__ __device__ inline int64_t first_group(int64_t place) { return 2 * place / (kGroup + 1); }

struct Order {
  int* start;        // [V + 1]: the rows of id v are rows[start[v] .. start[v + 1] - 1]
  int* rows;         // [N], ascending within an id
  int4* groups;      // {first place in rows, number of rows (0: none), first group of the id, id}
  int* summed;       // [groups, column blocks]: groups summed, counted at an id's first group
  float* sums;       // [groups, ld_sums]
  int64_t ld_sums;
};

// Sum over the block and this thread's exclusive prefix, of one int a thread.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// Latency: 12 us for 16384 rows and 149 CTAs (two passes over the ids, of which the second finds
// its keys in shared memory, and two over the 32 warps' counts), 6 for 255 rows.
__global__ void __launch_bounds__(kSortIds, 1)
    embed_sort_kernel(const int64_t* __restrict__ ids, int64_t ids_stride, int N, int V,
                      Order o, int max_groups, int col_blocks) {
  extern __shared__ int count[];      // [kSortWarps][kSortIds], then the keys of kSortKeys rows
  __shared__ int warp_sums[32];
  __shared__ int2 heavy[kSortIds];    // {id - lo, first group}
  __shared__ int n_heavy;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int lo = blockIdx.x * kSortIds;
  const int hi = min(lo + kSortIds, V);
  uint16_t* keys = reinterpret_cast<uint16_t*>(count + kSortWarps * kSortIds);
  const bool kept = N <= kSortKeys;
#pragma unroll 8
  for (int w = 0; w < kSortWarps; ++w) count[w * kSortIds + t] = 0;
  if (t == 0) n_heavy = 0;
  __syncthreads();
  griddep_wait();
  if (t == 0) griddep_launch_dependents();
  // each warp takes one stretch of the rows, a multiple of 32 long
  const int per = (int)((((int64_t)N + kSortIds - 1) / kSortIds) * 32);
  const int64_t n0 = (int64_t)warp * per;
  const int n1 = (int)(n0 + per < N ? n0 + per : N);
  int below = 0;
  int* mine = count + warp * kSortIds;
#pragma unroll 8
  for (int64_t n = n0 + lane; n < n1; n += 32) {
    const int64_t id = __ldg(ids + n * ids_stride);
    const bool own = id >= lo && id < hi;
    below += id >= 0 && id < lo;
    if (kept) keys[n] = own ? (uint16_t)(id - lo) : kNoKey;
    if (own) atomicAdd(mine + (int)(id - lo), 1);
  }
  int before, total, rows = 0;
  block_prefix(below, warp_sums, &before);      // rows with smaller ids; also a barrier
#pragma unroll 8
  for (int w = 0; w < kSortWarps; ++w) rows += count[w * kSortIds + t];
  int at = before + block_prefix(rows, warp_sums, &total);
  if (lo + t < V && RLK_STORE_OK(lo + t < V, &g_err_embedding)) {
    o.start[lo + t] = at;
    if (lo + t == V - 1) o.start[V] = at + rows;
    if (rows > kGroup) heavy[atomicAdd(&n_heavy, 1)] = make_int2(t, (int)first_group(at));
  }
  const int first = at;
#pragma unroll 8
  for (int w = 0; w < kSortWarps; ++w) {        // where each warp's rows of this id begin
    const int c = count[w * kSortIds + t];
    count[w * kSortIds + t] = at;
    at += c;
  }
  __syncthreads();
  // place the rows, in order within a warp
  for (int64_t n = n0 + lane; n - lane < n1; n += 32) {
    int key = -1;
    if (n < n1) {
      if (kept) {
        key = keys[n] == kNoKey ? -1 : keys[n];
      } else {
        const int64_t id = __ldg(ids + n * ids_stride);
        key = id >= lo && id < hi ? (int)(id - lo) : -1;
      }
    }
    const bool own = key >= 0;
    if (!__ballot_sync(0xffffffffu, own)) continue;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (own) {
      const int place = mine[key] + rank;
      if (RLK_STORE_OK(place >= 0 && place < N, &g_err_embedding)) o.rows[place] = (int)n;
    }
    __syncwarp();
    if (own && rank == 0) mine[key] += __popc(same);
    __syncwarp();
  }
  // the groups: those from this CTA's places on are its to clear (the last CTA's reach to the end),
  // and to fill for its ids with many rows; `first` of an id is what its thread computed
  const int clear_to =
      lo + kSortIds >= V ? max_groups : (int)first_group((int64_t)before + total);
  for (int g = (int)first_group(before) + t; g < clear_to; g += kSortIds)
    if (RLK_STORE_OK(g < max_groups, &g_err_embedding)) {
      o.groups[g] = make_int4(0, 0, 0, 0);
      for (int k = 0; k < col_blocks; ++k) o.summed[(int64_t)g * col_blocks + k] = 0;
    }
  __syncthreads();
  int* first_of = count;              // reused: every place was taken above
  int* rows_of = count + kSortIds;
  first_of[t] = first;
  rows_of[t] = rows;
  __syncthreads();
  for (int h = 0; h < n_heavy; ++h) {
    const int k = heavy[h].x, base = heavy[h].y;
    const int f = first_of[k], n = rows_of[k];
    const int groups = (n + kGroup - 1) / kGroup;    // a row past n may not fit an int, a group does
    for (int g = t; g < groups; g += kSortIds)
      if (RLK_STORE_OK(base + g < max_groups, &g_err_embedding))
        o.groups[base + g] =
            make_int4(f + g * kGroup, min(kGroup, n - g * kGroup), base, lo + k);
  }
}

// ---------------------------------------------------------------- gradient: the sums
// acc = the rows rows[at .. at + n - 1] of d at columns c + i * gap, added in that order, kDepth
// rows' loads in flight.
template <bool kFp32, int kRun, int kDepth>
__device__ __forceinline__ void add_rows(const void* __restrict__ d, int64_t ldd,
                                         const int* __restrict__ rows, int at, int n, int c,
                                         int gap, int H, float (&acc)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  int k = 0;
  for (; k + kDepth <= n; k += kDepth) {
    float v[kDepth][8];
#pragma unroll
    for (int j = 0; j < kDepth; ++j)
      load8<kFp32, kRun>(d, (int64_t)__ldg(rows + at + k + j) * ldd, c, gap, H, v[j]);
#pragma unroll
    for (int j = 0; j < kDepth; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[j][i]);
  }
#pragma unroll 2
  for (; k < n; ++k) {
    float v[8];
    load8<kFp32, kRun>(d, (int64_t)__ldg(rows + at + k) * ldd, c, gap, H, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[i]);
  }
}

// Sums of groups, which other blocks of this launch wrote.
template <int kRun>
__device__ __forceinline__ void load_sums(const float* s, int c, int gap, int H, float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / kRun; ++q) {
    const int k = c + q * gap;
    float* y = x + q * kRun;
#pragma unroll
    for (int j = 0; j < kRun; ++j) y[j] = 0.f;
    if (k >= H) continue;
    if constexpr (kRun == 1) {
      y[0] = __ldcg(s + k);
    } else {
#pragma unroll
      for (int j = 0; j < kRun; j += 4) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(s + k + j));
        y[j] = a.x; y[j + 1] = a.y; y[j + 2] = a.z; y[j + 3] = a.w;
      }
    }
  }
}

struct TableOut {
  void* dw;
  int64_t ldw;
  float scale;
  int H, V;
};

// A table row's eight columns from their sum.
template <bool kOutFp32, bool kAccumulate, int kRun>
__device__ __forceinline__ void write_row(const TableOut& out, int64_t v, int c, int gap,
                                          float (&acc)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = __fmul_rn(acc[i], out.scale);
  if (kAccumulate) {
    const float* p = static_cast<const float*>(out.dw) + v * out.ldw;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + run_at<kRun>(i, gap) < out.H)
        acc[i] = __fadd_rn(p[c + run_at<kRun>(i, gap)], acc[i]);
  }
  if (RLK_STORE_OK(v < out.V && min(c + run_at<kRun>(7, gap) + 1, out.H) <= out.ldw,
                   &g_err_embedding))
    store8<kOutFp32, kRun, true>(out.dw, v * out.ldw, c, gap, out.H, acc);
}

// The groups, by blocks of column steps: block b of group_blocks takes column step b / across and
// every across-th round of groups, most of them empty.  Latency (64 rows' loads, eight at a time),
// under the table's zeros.
template <bool kDFp32, bool kOutFp32, bool kAccumulate, int kRun>
__device__ __forceinline__ void sum_groups(const void* __restrict__ d, int64_t ldd, const Order& o,
                                           int max_groups, int across, int col_blocks,
                                           const TableOut& out, const RowLanes<kRun>& lanes) {
  __shared__ bool last[kRowThreads / 4];
  const int gap = lanes.gap(), row = lanes.row();
  const int by = (int)blockIdx.x / across, bx = (int)blockIdx.x - by * across;
  const int c = by * lanes.step() + lanes.col();
  for (int g0 = bx * lanes.rows(); g0 < max_groups; g0 += across * lanes.rows()) {
    const int g = g0 + row;
    const int4 what = g < max_groups ? o.groups[g] : make_int4(0, 0, 0, 0);
    const bool in = what.y > 0;
    if (!__syncthreads_or(in)) continue;
    float acc[8];
    if (in && c < out.H) {
      add_rows<kDFp32, kRun, kRun == 1 ? 2 : kDFp32 ? 4 : 8>(d, ldd, o.rows, what.x, what.y, c, gap,
                                                             out.H, acc);
      if (RLK_STORE_OK(g < max_groups && min(c + run_at<kRun>(7, gap) + 1, out.H) <= o.ld_sums,
                       &g_err_embedding))
        store8<true, kRun>(o.sums, g * o.ld_sums, c, gap, out.H, acc);
    }
    __threadfence();
    __syncthreads();
    int groups = 0;
    if (in) groups = (o.start[what.w + 1] - o.start[what.w] + kGroup - 1) / kGroup;
    if (in && lanes.col() == 0)
      last[row] = atomicAdd(o.summed + (int64_t)what.z * col_blocks + by, 1) == groups - 1;
    __syncthreads();
    if (in && last[row] && c < out.H) {
      __threadfence();
      const float* s = o.sums + (int64_t)what.z * o.ld_sums;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
      for (int k = 0; k < groups; ++k) {
        float x[8];
        load_sums<kRun>(s + k * o.ld_sums, c, gap, out.H, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], x[i]);
      }
      write_row<kOutFp32, kAccumulate, kRun>(out, what.w, c, gap, acc);
    }
  }
}

// Threads of a row take `turns` (at most kRowsInTurn) consecutive table rows, most of them rows of
// zeros: how many rows of d each has is read for all of them at once, and the zeros wait for
// nothing.  Written past the caches (nothing reads a table's gradient soon: 47 against 51 us for a
// lookup and gradient of 32003 x 2048 FP32).  Bound by HBM: 151936 x 4096 BF16 from 16384 rows 220
// us (1.32 GB, 6.0 TB/s; 377 with a block a row, and 13 more for the groups in a launch of their
// own), that FP32 table 40 (6.6 TB/s).
constexpr int kRowsInTurn = 16;

template <bool kDFp32, bool kOutFp32, bool kAccumulate, int kRun>
__global__ void __launch_bounds__(kRowThreads, 4)
    embed_rows_kernel(const void* __restrict__ d, int64_t ldd, Order o, int max_groups,
                      int group_blocks, int across, TableOut out, int turns, RowLanes<kRun> lanes) {
  __shared__ int start[kRowThreads / 4 * kRowsInTurn + 1];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if ((int)blockIdx.x < group_blocks) {
    sum_groups<kDFp32, kOutFp32, kAccumulate, kRun>(d, ldd, o, max_groups, across,
                                                    group_blocks / across, out, lanes);
    return;
  }
  const int V = out.V, H = out.H;
  const int per_block = lanes.rows() * turns;
  const int64_t first = (int64_t)(blockIdx.x - group_blocks) * per_block;
  for (int i = threadIdx.x; i <= per_block; i += kRowThreads)
    start[i] = __ldg(o.start + (first + i < V ? first + i : V));
  __syncthreads();
  const int gap = lanes.gap();
#pragma unroll 1
  for (int k = 0; k < turns; ++k) {
    const int mine = lanes.row() * turns + k;
    const int64_t v = first + mine;
    if (v >= V) break;
    const int at = start[mine], n = start[mine + 1] - at;
    if (n > kGroup || (kAccumulate && n == 0)) continue;
    for (int c = lanes.col(); c < H; c += lanes.step()) {
      float acc[8];
      add_rows<kDFp32, kRun, kRun == 1 ? 2 : 4>(d, ldd, o.rows, at, n, c, gap, H, acc);
      write_row<kOutFp32, kAccumulate, kRun>(out, v, c, gap, acc);
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxWidth = int64_t(1) << 20;
// ids of a gradient: a sorting CTA's last + 1 fits an int
constexpr int64_t kMaxTable = int64_t(1) << 30;
// Every sorting CTA reads all ids: 2^37 reads are about a second with a CTA on every SM (2^20 rows
// of a table of 2^27).  A small table has few of them: 2^24 rows of 1000 ids, one CTA, take 22 ms.
constexpr int64_t kMaxSortReads = int64_t(1) << 37;

struct EmbedPlan {
  int64_t groups = 0, ld_sums = 0;
  size_t off_rows = 0, off_groups = 0, off_summed = 0, off_sums = 0, total = 0;
};

// Column steps of a pass: at most 256 threads of eight columns a row (at least four threads).
inline int64_t column_steps(int64_t H) { return ceil_div(H, 8 * kRowThreads); }

bool embed_plan(int64_t N, int64_t V, int64_t H, EmbedPlan* p) {
  if (N < 0 || N >= kMaxExtent || V < 1 || V >= kMaxTable || H < 1 || H >= kMaxWidth ||
      N * ceil_div(V, kSortIds) >= kMaxSortReads)
    return false;
  p->groups = first_group(N);
  p->ld_sums = ceil_div(H, 8) * 8;
  size_t off = align_up((size_t)(V + 1) * 4, 256);
  p->off_rows = off;
  off = align_up(off + (size_t)N * 4, 256);
  p->off_groups = off;
  off = align_up(off + (size_t)p->groups * 16, 256);
  p->off_summed = off;
  off = align_up(off + (size_t)p->groups * column_steps(H) * 4, 256);
  p->off_sums = off;
  p->total = align_up(off + (size_t)p->groups * p->ld_sums * 4, 256);
  return true;
}

// The run length (see RowLanes) that both matrices of a pass allow: by the output's type, or 1.
int embed_run(int64_t H, const void* in, int in_dtype, int64_t ld_in, const void* out,
              int out_dtype, int64_t ld_out) {
  const int n = out_dtype == RLK_FP32 ? 4 : 8;
  return rows_vec(in, ld_in, dtype_bytes(in_dtype), H, n) &&
                 rows_vec(out, ld_out, dtype_bytes(out_dtype), H, n)
             ? n
             : 1;
}
template <class Out32, class F>
cudaError_t by_run(int run, Out32, F f) {
  return run == 1 ? f(Const<1>()) : f(Const<Out32::value ? 4 : 8>());
}

std::mutex g_attr_mutex;
bool g_attr_set[64];

cudaError_t ensure_attrs(int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!g_attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem(kSortKeys));
    if (e != cudaSuccess) return e;
    g_attr_set[dev] = true;
  }
  return cudaSuccess;
}

rlk_status cuda_failed() {
  cudaGetLastError();
  return RLK_ERR_CUDA;
}

}  // namespace

uint32_t take_error_embedding() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_embedding, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaMemcpyToSymbol(g_err_embedding, &zero, sizeof zero);
  cudaGetLastError();
  return v;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_embedding(const int64_t* ids, int64_t ids_stride, int64_t N, const void* weight,
                         int weight_dtype, int64_t V, int64_t H, int64_t ld_weight, float scale,
                         void* out, int out_dtype, int64_t ld_out, void* stream) {
  RLK_CALL_RANGE();
  if (!known_dtype(weight_dtype) || !known_dtype(out_dtype)) return RLK_ERR_DTYPE;
  if (N < 0 || N >= kMaxExtent || V < 1 || V >= kMaxExtent || H < 1 || H >= kMaxWidth ||
      ids_stride < 0 || ids_stride >= kPitchLimit || ld_weight < H || ld_weight >= kPitchLimit ||
      ld_out < H || ld_out >= kPitchLimit)
    return RLK_ERR_SHAPE;
  if (!isfinite(scale)) return RLK_ERR_VALUE;
  if (N == 0) return RLK_OK;
  if (!ids || !weight || !out) return RLK_ERR_NULL;
  if (!is_aligned(ids, 8) || !is_aligned(weight, dtype_bytes(weight_dtype)) ||
      !is_aligned(out, dtype_bytes(out_dtype)))
    return RLK_ERR_ALIGN;
  DeviceInfo dev;
  const rlk_status st = device_ready(&dev);
  if (st != RLK_OK) return st;
  const int run = embed_run(H, weight, weight_dtype, ld_weight, out, out_dtype, ld_out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = by_dtypes(weight_dtype, out_dtype, [&](auto w32, auto o32) {
    return by_run(run, o32, [&](auto r) {
      constexpr int kRun = decltype(r)::value;
      const RowLanes<kRun> lanes = row_lanes<kRun>(H);
      const dim3 grid((unsigned)ceil_div(N, lanes.rows()));
      return launch_overlapped(embed_kernel<decltype(w32)::value, decltype(o32)::value, kRun>, grid,
                               kRowThreads, 0, s, ids, ids_stride, N, weight, V, (int)H, ld_weight,
                               scale, out, ld_out, lanes);
    });
  });
  return e == cudaSuccess ? RLK_OK : cuda_failed();
}

size_t rlk_embedding_backward_workspace_size(int64_t N, int64_t V, int64_t H) {
  EmbedPlan p;
  return embed_plan(N, V, H, &p) ? p.total : 0;
}

rlk_status rlk_embedding_backward(const int64_t* ids, int64_t ids_stride, int64_t N,
                                  const void* grad, int grad_dtype, int64_t H, int64_t ld_grad,
                                  float scale, void* grad_weight, int grad_weight_dtype, int64_t V,
                                  int64_t ld_grad_weight, int accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  RLK_CALL_RANGE();
  if (!known_dtype(grad_dtype) || !known_dtype(grad_weight_dtype) ||
      (accumulate && grad_weight_dtype != RLK_FP32))
    return RLK_ERR_DTYPE;
  EmbedPlan p;
  if (!embed_plan(N, V, H, &p) || ids_stride < 0 || ids_stride >= kPitchLimit || ld_grad < H ||
      ld_grad >= kPitchLimit || ld_grad_weight < H || ld_grad_weight >= kPitchLimit)
    return RLK_ERR_SHAPE;
  if (!isfinite(scale)) return RLK_ERR_VALUE;
  if (N == 0 && accumulate) return RLK_OK;
  if (!grad_weight || (N > 0 && (!ids || !grad))) return RLK_ERR_NULL;
  const size_t esize = dtype_bytes(grad_weight_dtype);
  if (!is_aligned(ids, 8) || !is_aligned(grad, dtype_bytes(grad_dtype)) ||
      !is_aligned(grad_weight, esize))
    return RLK_ERR_ALIGN;
  if (N > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < p.total))
    return RLK_ERR_WORKSPACE;
  DeviceInfo dev;
  const rlk_status st = device_ready(&dev);
  if (st != RLK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0)
    return cudaMemset2DAsync(grad_weight, ld_grad_weight * esize, 0, H * esize, V, s) == cudaSuccess
               ? RLK_OK
               : cuda_failed();
  if (ensure_attrs(dev.device) != cudaSuccess) return cuda_failed();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Order o;
  o.start = reinterpret_cast<int*>(ws);
  o.rows = reinterpret_cast<int*>(ws + p.off_rows);
  o.groups = reinterpret_cast<int4*>(ws + p.off_groups);
  o.summed = reinterpret_cast<int*>(ws + p.off_summed);
  o.sums = reinterpret_cast<float*>(ws + p.off_sums);
  o.ld_sums = p.ld_sums;
  if (launch_overlapped(embed_sort_kernel, dim3((unsigned)ceil_div(V, kSortIds)), kSortIds,
                        sort_smem(N), s, ids, ids_stride, (int)N, (int)V, o,
                        (int)p.groups, (int)column_steps(H)) != cudaSuccess)
    return cuda_failed();
  const int run = embed_run(H, grad, grad_dtype, ld_grad, grad_weight, grad_weight_dtype,
                            ld_grad_weight);
  const cudaError_t e = by_dtypes(grad_dtype, grad_weight_dtype, [&](auto d32, auto o32) {
    return by_run(run, o32, [&](auto r) {
      constexpr bool kD = decltype(d32)::value, kO = decltype(o32)::value;
      constexpr int kRun = decltype(r)::value;
      const RowLanes<kRun> lanes = row_lanes<kRun>(H);
      // the groups' blocks: four an SM, or all there can be
      const int64_t col_blocks = ceil_div(H, lanes.step());     // column_steps(H)
      int64_t across = ceil_div(4 * (int64_t)dev.sm_count, col_blocks);
      const int64_t all = N > kGroup ? ceil_div(p.groups, lanes.rows()) : 0;
      if (across > all) across = all;
      // 16 table rows in turn a row of threads, fewer where that leaves under 16 blocks an SM
      int turns = kRowsInTurn;
      while (turns > 1 && ceil_div(V, lanes.rows() * turns) < 16 * dev.sm_count) turns /= 2;
      const int64_t group_blocks = across * col_blocks;
      const dim3 grid((unsigned)(group_blocks + ceil_div(V, lanes.rows() * turns)));
      const TableOut out = {grad_weight, ld_grad_weight, scale, (int)H, (int)V};
      if constexpr (kO)
        if (accumulate)
          return launch_overlapped(embed_rows_kernel<kD, true, true, kRun>, grid, kRowThreads, 0, s,
                                   grad, ld_grad, o, (int)p.groups, (int)group_blocks, (int)across,
                                   out, turns, lanes);
      return launch_overlapped(embed_rows_kernel<kD, kO, false, kRun>, grid, kRowThreads, 0, s,
                               grad, ld_grad, o, (int)p.groups, (int)group_blocks, (int)across, out,
                               turns, lanes);
    });
  });
  return e == cudaSuccess ? RLK_OK : cuda_failed();
}

}  // extern "C"
