// Pages of paged caches, managed on the device: which sequences hold which page (reference counts),
// the block table, and the moves of page contents in every layer's arrays.
//
// All results are functions of the state at entry: free pages are taken in ascending order by
// (sequence, logical page), moves pair the highest live pages with the lowest holes, and the only
// atomics are integer additions to reference counts. A call that cannot be carried out in full
// changes nothing and says so in *status.
//
// The plan of a call (rank of every free or live page) is one launch of a cluster of 8 CTAs: each
// warp counts its contiguous 1/256 of the reference counts, the CTA totals are exchanged through
// distributed shared memory, and a second pass over the same (now cached) counts hands out ranks.
// It is bound by launch and latency: a pool of 64 K pages is 256 KB of counts. Page contents move
// as 16-byte vectors, 8 KB units flattened over (page, array) so that the small arrays of a page
// do not leave CTAs idle; bound by HBM.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kSeqPer = kMaxPoolB / kPlanThreads; // sequences a thread of a plan owns
constexpr int kCopyThreads = 128;
constexpr int kCopyVecs = 4; // 16-byte vectors a thread moves at a time
constexpr unsigned kChunk = kCopyThreads * kCopyVecs * 16;

enum { kExtend, kFork, kCompact };

// Workspace of fork and compact calls (int32):
//   fork:    state, then for each sequence its parent or -1, the new length and the fresh page or
//            -1, then the new block-table rows (the parent's partial page still in place)
//   compact: number of moves, then for each k the source and the hole of move k, then for each
//            page at or above the live count its move or -1
struct ForkWs {
  int *state, *parent, *len, *fresh, *rows;
  __host__ __device__ ForkWs(void *ws, int B)
      : state(static_cast<int *>(ws)), parent(state + 4), len(parent + B), fresh(len + B), rows(fresh + B) {}
};
struct CompactWs {
  int *moves, *src, *hole, *move_of;
  __host__ __device__ CompactWs(void *ws, int pages)
      : moves(static_cast<int *>(ws)), src(moves + 4), hole(src + pages), move_of(hole + pages) {}
};

__device__ __forceinline__ int pages_for(int len, int page_size) {
  return (len + page_size - 1) / page_size; // len <= max_pages * page_size <= 2^30
}

struct PlanArgs {
  tq_page_pool p;
  const int *in; // extend: positions to add; fork: parents
  int *status;   // extend, fork
  int *live;     // compact
  void *ws;
};

// Inclusive scan over the CTA's threads; every thread gets its prefix and the total.
__device__ __forceinline__ int block_scan(int v, int *s_warp, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  return before + v;
}

template <int MODE>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int s_pre[MODE == kCompact ? 1 : kMaxPoolB]; // pages handed to the sequences before this one
  __shared__ int s_had[MODE == kExtend ? kMaxPoolB : 1];  // pages the sequence had
  __shared__ int s_warp[kPlanWarps];
  __shared__ int s_total; // this CTA's count, read by the others
  __shared__ int s_long; // a sequence would pass its row of the table
  __shared__ unsigned long long s_sum;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster.block_rank();
  const int B = a.p.B, ps = a.p.page_size, pages = a.p.num_pages, cap = a.p.max_pages * ps;
  pdl_wait();
  if (tid == 0) s_long = 0, s_sum = 0;
  __syncthreads();
  // ---- what each sequence needs (every CTA computes all of it)
  int wanted = 0;
  if constexpr (MODE != kCompact) {
    ForkWs f(a.ws, B);
    int need[kSeqPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kSeqPer; ++i) {
      const int b = tid * kSeqPer + i;
      need[i] = 0;
      if (b >= B) continue;
      if constexpr (MODE == kExtend) {
        const int len = max(a.p.lens[b], 0);
        const long long after = static_cast<long long>(len) + max(a.in[b], 0);
        if (after > cap) s_long = 1;
        else need[i] = pages_for(static_cast<int>(after), ps) - pages_for(len, ps);
        s_had[b] = len <= cap ? pages_for(len, ps) : 0;
      } else {
        const int par = a.in[b];
        const bool valid = par >= 0 && par < B && par != b;
        const int len = valid ? min(max(a.p.lens[par], 0), cap) : 0;
        need[i] = len % ps != 0;
        if (rank == 0) f.parent[b] = valid ? par : -1, f.len[b] = len, f.fresh[b] = -1;
      }
      sum += need[i]; // at most 4 * 2^26
    }
    const int incl = block_scan(sum, s_warp, wanted);
    atomicAdd(&s_sum, static_cast<unsigned long long>(sum)); // the scan itself may wrap; then the call fails
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < kSeqPer; ++i) {
      const int b = tid * kSeqPer + i;
      if (b < B) s_pre[b] = run;
      run += need[i];
    }
  }
  // ---- count the free (compact: live) pages of this warp's part of the pool
  const int part = ((pages + kCluster * kPlanWarps - 1) / (kCluster * kPlanWarps) + 127) / 128 * 128;
  const long long begin = static_cast<long long>(rank * kPlanWarps + warp) * part;
  const int lo = static_cast<int>(min(begin, static_cast<long long>(pages)));
  const int hi = static_cast<int>(min(begin + part, static_cast<long long>(pages)));
  auto load = [&](int i, bool (&hit)[4]) { // pages i .. i + 3 (i a multiple of 4)
    int r[4] = {1, 1, 1, 1};
    if (i + 4 <= pages) {
      const int4 v = *reinterpret_cast<const int4 *>(a.p.refs + i);
      r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else {
      for (int e = 0; e < 4; ++e)
        if (i + e < pages) r[e] = a.p.refs[i + e];
    }
    for (int e = 0; e < 4; ++e) hit[e] = i + e < pages && (MODE == kCompact ? r[e] != 0 : r[e] == 0);
  };
  int cnt = 0;
  for (int i = lo + lane * 4; i < hi; i += 128) {
    bool hit[4];
    load(i, hit);
#pragma unroll
    for (int e = 0; e < 4; ++e) cnt += hit[e];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  __syncthreads(); // block_scan's readers of s_warp are done
  if (lane == 0) s_warp[warp] = cnt;
  __syncthreads();
  if (tid == 0) {
    int t = 0;
    for (int w = 0; w < kPlanWarps; ++w) t += s_warp[w];
    s_total = t;
  }
  cluster.sync(); // totals are visible; every CTA has read lens and its part of refs
  int before = 0, all = 0;
  for (int r = 0; r < kCluster; ++r) {
    const int t = *cluster.map_shared_rank(&s_total, r);
    if (r < rank) before += t;
    all += t;
  }
  cluster.sync(); // nobody leaves while its total is being read
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  if constexpr (MODE != kCompact) {
    const int status = s_long ? 2 : s_sum > static_cast<unsigned long long>(all) ? 1 : 0;
    if (rank == 0 && tid == 0) {
      *a.status = status;
      if constexpr (MODE == kFork) ForkWs(a.ws, B).state[0] = status;
    }
    if (status != 0) return;
  }
  if constexpr (MODE == kCompact) {
    if (rank == 0 && tid == 0) {
      *a.live = all;
      if (all == pages) *CompactWs(a.ws, pages).moves = 0;
    }
  }
  // ---- hand out the ranks
  for (int i0 = lo; i0 < hi; i0 += 128) {
    if (MODE != kCompact && before >= wanted) break;
    const int i = i0 + lane * 4;
    bool hit[4] = {false, false, false, false};
    if (i < hi) load(i, hit);
    int sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += hit[e];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    int k = before + incl - sum; // free (live) pages before this one
    before += __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int page = i + e;
      if constexpr (MODE == kCompact) {
        if (page >= pages || i >= hi) continue;
        CompactWs c(a.ws, pages);
        if (page == all) *c.moves = all - k;
        if (page < all) {
          if (!hit[e]) c.hole[page - k] = page;
        } else {
          const int m = all - 1 - k; // live pages above this one
          if (hit[e]) c.src[m] = page;
          c.move_of[page] = hit[e] ? m : -1;
        }
        k += hit[e];
      } else {
        if (hit[e] && k < wanted) {
          int b0 = 0, b1 = B; // the last sequence with s_pre <= k
          while (b1 - b0 > 1) {
            const int mid = (b0 + b1) >> 1;
            (s_pre[mid] <= k ? b0 : b1) = mid;
          }
          if constexpr (MODE == kExtend)
            a.p.block_table[static_cast<long long>(b0) * a.p.max_pages + s_had[b0] + (k - s_pre[b0])] = page;
          else
            ForkWs(a.ws, B).fresh[b0] = page;
          a.p.refs[page] = 1;
        }
        k += hit[e];
      }
    }
  }
  if (MODE == kExtend && rank == 0) { // every CTA has read lens (first cluster barrier)
    for (int b = tid; b < B; b += kPlanThreads) a.p.lens[b] = max(a.p.lens[b], 0) + max(a.in[b], 0);
  }
}

// ---------------------------------------------------------------- page contents
template <int N>
struct Arrays {
  struct {
    uint8_t *base;
    unsigned bytes, first; // bytes of a page, 8 KB units of the arrays before this one
  } a[N];
  int n;
  unsigned units; // 8 KB units of a page over all arrays
};

template <int N>
__device__ __forceinline__ void move_unit(const Arrays<N> &ar, unsigned unit, int src, int dst) {
  int lo = 0, hi = ar.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    (ar.a[mid].first <= unit ? lo : hi) = mid;
  }
  const size_t bytes = ar.a[lo].bytes;
  const unsigned at = (unit - ar.a[lo].first) * kChunk + threadIdx.x * 16;
  const uint8_t *s = ar.a[lo].base + bytes * src + at;
  uint8_t *d = ar.a[lo].base + bytes * dst + at;
  uint4 v[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + i * kCopyThreads * 16 < bytes) v[i] = *reinterpret_cast<const uint4 *>(s + i * kCopyThreads * 16);
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + i * kCopyThreads * 16 < bytes) *reinterpret_cast<uint4 *>(d + i * kCopyThreads * 16) = v[i];
}

struct Pairs {
  int src[kPageCopyBatch], dst[kPageCopyBatch];
  int n;
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ Arrays<N> ar,
                                                            const __grid_constant__ Pairs pairs) {
  pdl_wait();
  const unsigned long long work = static_cast<unsigned long long>(pairs.n) * ar.units;
  for (unsigned long long w = blockIdx.x; w < work; w += gridDim.x) {
    const unsigned m = static_cast<unsigned>(w / ar.units);
    move_unit(ar, static_cast<unsigned>(w - static_cast<unsigned long long>(m) * ar.units), pairs.src[m], pairs.dst[m]);
  }
}

// ---------------------------------------------------------------- fork
// The new rows, from the table as it was, and the children's old pages given back.
__global__ void __launch_bounds__(256) fork_rows_kernel(const tq_page_pool p, void *ws) {
  pdl_wait();
  ForkWs f(ws, p.B);
  if (f.state[0] != 0) return;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int par = f.parent[b];
    if (par < 0) continue;
    const int n = pages_for(f.len[b], p.page_size);
    const long long row = static_cast<long long>(b) * p.max_pages;
    for (int j = blockIdx.x * 256 + threadIdx.x; j < p.max_pages; j += gridDim.x * 256) {
      const int old = p.block_table[row + j];
      if (old >= 0 && old < p.num_pages) atomicSub(p.refs + old, 1);
      f.rows[row + j] = j < n ? p.block_table[static_cast<long long>(par) * p.max_pages + j] : -1;
    }
  }
}

// Blocks of y = 0 write the table, lengths and counts; those of y = 1 copy the partial pages.
template <int N>
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const tq_page_pool p,
                                                                  const __grid_constant__ Arrays<N> ar, void *ws) {
  pdl_wait();
  ForkWs f(ws, p.B);
  if (f.state[0] != 0) return;
  if (blockIdx.y == 0) {
    const int across = (p.max_pages + kCopyThreads - 1) / kCopyThreads;
    for (long long w = blockIdx.x; w < static_cast<long long>(across) * p.B; w += gridDim.x) {
      const int b = static_cast<int>(w / across), j = static_cast<int>(w - static_cast<long long>(b) * across) * kCopyThreads + threadIdx.x;
      if (f.parent[b] < 0 || j >= p.max_pages) continue;
      const long long row = static_cast<long long>(b) * p.max_pages;
      const int fresh = f.fresh[b], len = f.len[b];
      int e = f.rows[row + j];
      if (fresh >= 0 && j == len / p.page_size) e = fresh; // counted when it was handed out
      else if (e >= 0 && e < p.num_pages) atomicAdd(p.refs + e, 1);
      p.block_table[row + j] = e;
      if (j == 0) p.lens[b] = len;
    }
    return;
  }
  for (long long w = blockIdx.x; w < static_cast<long long>(p.B) * ar.units; w += gridDim.x) {
    const int b = static_cast<int>(w / ar.units);
    const int fresh = f.fresh[b];
    if (fresh < 0) continue;
    const int src = f.rows[static_cast<long long>(b) * p.max_pages + f.len[b] / p.page_size];
    if (src < 0 || src >= p.num_pages) continue;
    move_unit(ar, static_cast<unsigned>(w - static_cast<long long>(b) * ar.units), src, fresh);
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(256) free_kernel(const tq_page_pool p, const int *leaving) {
  pdl_wait();
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    if (leaving[b] == 0) continue;
    const long long row = static_cast<long long>(b) * p.max_pages;
    for (int j = blockIdx.x * 256 + threadIdx.x; j < p.max_pages; j += gridDim.x * 256) {
      const int e = p.block_table[row + j];
      if (e >= 0 && e < p.num_pages) atomicSub(p.refs + e, 1);
      p.block_table[row + j] = -1;
      if (j == 0) p.lens[b] = 0;
    }
  }
}

// ---------------------------------------------------------------- compact
template <int N>
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const tq_page_pool p,
                                                                     const __grid_constant__ Arrays<N> ar,
                                                                     const int *live, void *ws) {
  pdl_wait();
  CompactWs c(ws, p.num_pages);
  const int moves = *c.moves;
  if (moves == 0) return;
  const int n = *live;
  if (blockIdx.y == 0) {
    const long long entries = static_cast<long long>(p.B) * p.max_pages, step = static_cast<long long>(gridDim.x) * kCopyThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries; i += step) {
      const int e = p.block_table[i];
      if (e < n || e >= p.num_pages) continue;
      const int m = c.move_of[e];
      if (m >= 0) p.block_table[i] = c.hole[m];
    }
    for (long long m = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; m < moves; m += step) {
      p.refs[c.hole[m]] = p.refs[c.src[m]];
      p.refs[c.src[m]] = 0;
    }
    return;
  }
  for (long long w = blockIdx.x; w < static_cast<long long>(moves) * ar.units; w += gridDim.x) {
    const int m = static_cast<int>(w / ar.units);
    move_unit(ar, static_cast<unsigned>(w - static_cast<long long>(m) * ar.units), c.src[m], c.hole[m]);
  }
}

// ---------------------------------------------------------------- launches
template <int N>
Arrays<N> pack(const tq_page_array *arrays, int n) {
  Arrays<N> ar;
  ar.n = n;
  ar.units = 0;
  for (int i = 0; i < n; ++i) {
    ar.a[i].base = static_cast<uint8_t *>(arrays[i].base);
    ar.a[i].bytes = static_cast<unsigned>(arrays[i].page_bytes);
    ar.a[i].first = ar.units;
    ar.units += (ar.a[i].bytes + kChunk - 1) / kChunk;
  }
  return ar;
}

// Kernels that move pages take their arrays as launch parameters; one layer's few in a small
// block, many layers' in a large one.
constexpr int kFewArrays = 32;

template <class F>
cudaError_t with_arrays(const tq_page_array *arrays, int n, F &&f) {
  return n <= kFewArrays ? f(pack<kFewArrays>(arrays, n)) : f(pack<kMaxPageArrays>(arrays, n));
}

dim3 row_grid(const tq_page_pool &p) {
  return dim3(static_cast<unsigned>(std::min((p.max_pages + 255) / 256, 64)), static_cast<unsigned>(p.B));
}

} // namespace

size_t pages_workspace_bytes(const tq_page_pool &p) {
  const size_t fork = 4 + 3 * static_cast<size_t>(p.B) + static_cast<size_t>(p.B) * p.max_pages;
  const size_t compact = 4 + 3 * static_cast<size_t>(p.num_pages);
  return (std::max(fork, compact) * sizeof(int) + 15) / 16 * 16;
}

cudaError_t launch_pages_extend(const tq_page_pool &p, const int *need, int *status, cudaStream_t s) {
  return launch_pdl(plan_kernel<kExtend>, dim3(kCluster), dim3(kPlanThreads), 0, s,
                    PlanArgs{p, need, status, nullptr, nullptr});
}

cudaError_t launch_pages_fork(const tq_page_pool &p, const tq_page_array *arrays, int n_arrays,
                              const int *parent_of, int *status, void *ws, int sm_count, cudaStream_t s) {
  cudaError_t e = launch_pdl(plan_kernel<kFork>, dim3(kCluster), dim3(kPlanThreads), 0, s,
                             PlanArgs{p, parent_of, status, nullptr, ws});
  if (e != cudaSuccess) return e;
  e = launch_pdl(fork_rows_kernel, row_grid(p), dim3(256), 0, s, p, ws);
  if (e != cudaSuccess) return e;
  return with_arrays(arrays, n_arrays, [&](const auto &ar) {
    using A = std::decay_t<decltype(ar)>;
    constexpr int N = sizeof(A) > sizeof(Arrays<kFewArrays>) ? kMaxPageArrays : kFewArrays;
    return launch_pdl(fork_apply_kernel<N>, dim3(sm_count * 8, n_arrays ? 2 : 1), dim3(kCopyThreads), 0, s, p, ar, ws);
  });
}

cudaError_t launch_pages_free(const tq_page_pool &p, const int *leaving, cudaStream_t s) {
  return launch_pdl(free_kernel, row_grid(p), dim3(256), 0, s, p, leaving);
}

cudaError_t launch_pages_compact(const tq_page_pool &p, const tq_page_array *arrays, int n_arrays, int *live,
                                 void *ws, int sm_count, cudaStream_t s) {
  cudaError_t e = launch_pdl(plan_kernel<kCompact>, dim3(kCluster), dim3(kPlanThreads), 0, s,
                             PlanArgs{p, nullptr, nullptr, live, ws});
  if (e != cudaSuccess) return e;
  return with_arrays(arrays, n_arrays, [&](const auto &ar) {
    using A = std::decay_t<decltype(ar)>;
    constexpr int N = sizeof(A) > sizeof(Arrays<kFewArrays>) ? kMaxPageArrays : kFewArrays;
    return launch_pdl(compact_apply_kernel<N>, dim3(sm_count * 8, n_arrays ? 2 : 1), dim3(kCopyThreads), 0, s, p, ar,
                      static_cast<const int *>(live), ws);
  });
}

cudaError_t launch_pages_copy(const tq_page_array *arrays, int n_arrays, const int *src, const int *dst, int n,
                              int sm_count, cudaStream_t s) {
  return with_arrays(arrays, n_arrays, [&](const auto &ar) {
    using A = std::decay_t<decltype(ar)>;
    constexpr int N = sizeof(A) > sizeof(Arrays<kFewArrays>) ? kMaxPageArrays : kFewArrays;
    for (int at = 0; at < n; at += kPageCopyBatch) {
      Pairs pairs;
      pairs.n = std::min(kPageCopyBatch, n - at);
      std::copy(src + at, src + at + pairs.n, pairs.src);
      std::copy(dst + at, dst + at + pairs.n, pairs.dst);
      const unsigned long long work = static_cast<unsigned long long>(pairs.n) * ar.units;
      const unsigned grid = static_cast<unsigned>(std::min<unsigned long long>(work, sm_count * 12ull));
      const cudaError_t e = launch_pdl(copy_kernel<N>, dim3(grid), dim3(kCopyThreads), 0, s, ar, pairs);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  });
}

} // namespace tq
