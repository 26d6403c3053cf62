// Pages of paged caches, managed on the device: which sequences hold which page (reference counts),
// the block table, and the moves of page contents in every layer's arrays.
//
// All results are functions of the state at entry: free pages are taken in ascending order by
// (sequence, logical page), moves pair the highest live pages with the lowest holes, and the only
// atomics are integer additions to reference counts. A call that cannot be carried out in full
// changes nothing and says so in *status. (Extend first gives back pages that a caller left behind a
// length it lowered, in any case: kept, their entries would be written over and their counts lost.
// Seeing that there are none, by one entry of each sequence, costs an extend 0.3 to 0.6 us; loading the
// entries ahead of the counts was no faster.)
//
// Bookkeeping of a call is one launch of one cluster: 1 CTA for pools of up to 16 K pages, 8 above
// (extend and free of 32 sequences, one CTA against 8: 7.4 and 8.8 us for 1000 pages, 8.2 and 9.6 for 4096,
// 10.0 and 9.6 for 8192, 11.5 and 9.6 for 16384, 13.8 and 9.7 for 32768; compact 3.6 and 5.0, 4.5 and 6.0,
// 5.9 and 6.6, 8.5 and 6.7, 13.4 and 6.6). Each warp counts its contiguous
// share of the reference counts, the CTA totals are exchanged through distributed shared memory, and
// a second look at the same counts (held as a bit mask a lane) hands out ranks. It is bound by
// launch, memory latency and cold instructions, so its code is kept short. Page contents move as
// 16-byte vectors, 8 KB units flattened over (page, array) so that the small arrays of a page do not
// leave CTAs idle; bound by HBM.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;         // CTAs of a plan for a large pool
constexpr int kSmallPool = 1 << 14; // pages that one CTA plans
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr long long kSmallTable = 1 << 12; // table entries whose rows a fork's plan writes itself
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

struct PlanArgs {
  tq_page_pool p;
  int shift;     // log2(page size)
  const int *in; // extend: positions to add; fork: parents
  int *status;   // extend, fork
  int *granted;  // extend: positions added, or NULL; may be `in`
  int *live;     // compact
  void *ws;
  bool rows;     // fork, one CTA: the rows of the table too
};

__device__ __forceinline__ int pages_for(int len, int shift) { return (len + (1 << shift) - 1) >> shift; } // len <= 2^30

__device__ __forceinline__ bool is_page(const tq_page_pool &p, int e) { return static_cast<unsigned>(e) < static_cast<unsigned>(p.num_pages); }

// A warp gives back the pages of a row from entry j on, up to 32 entries without one.
__device__ __forceinline__ void give_back(const tq_page_pool &p, int b, int j, int lane) {
  int *row = p.block_table + static_cast<long long>(b) * p.max_pages;
  bool some = true;
#pragma unroll 1
  for (; some && j < p.max_pages; j += 32) {
    const int at = j + lane, e = at < p.max_pages ? row[at] : -1;
    if (is_page(p, e)) {
      atomicSub(p.refs + e, 1);
      row[at] = -1;
    }
    some = __any_sync(0xffffffffu, is_page(p, e));
  }
}

// A child's new row of the table, from the table as it was, and its old pages given back.
__device__ __forceinline__ void gather_row(const tq_page_pool &p, int shift, const ForkWs &f, int b, int from, int step) {
  const int par = f.parent[b];
  if (par < 0) return;
  const int n = pages_for(f.len[b], shift);
  const long long row = static_cast<long long>(b) * p.max_pages;
  for (int j = from; j < p.max_pages; j += step) {
    const int old = p.block_table[row + j];
    if (old >= 0 && old < p.num_pages) atomicSub(p.refs + old, 1);
    f.rows[row + j] = j < n ? p.block_table[static_cast<long long>(par) * p.max_pages + j] : -1;
  }
}
// Writes the row, its length and its counts.
__device__ __forceinline__ void apply_row(const tq_page_pool &p, int shift, const ForkWs &f, int b, int from, int step) {
  if (f.parent[b] < 0) return;
  const long long row = static_cast<long long>(b) * p.max_pages;
  const int fresh = f.fresh[b], len = f.len[b];
  for (int j = from; j < p.max_pages; j += step) {
    int e = f.rows[row + j];
    if (fresh >= 0 && j == len >> shift) e = fresh; // counted when it was handed out
    else if (e >= 0 && e < p.num_pages) atomicAdd(p.refs + e, 1);
    p.block_table[row + j] = e;
    if (j == 0) p.lens[b] = len;
  }
}

// Prefix of a thread's number over the CTA's threads (those before it) and the total.
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned *s_warp, unsigned &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads(); // the readers of the scan before are done
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  unsigned w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  return (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0u) + incl - v;
}

template <int MODE>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ unsigned s_pre[MODE == kCompact ? 1 : kMaxPoolB]; // pages handed to the sequences before this one
  __shared__ int s_had[MODE == kExtend ? kMaxPoolB : 1];       // pages the sequence had
  __shared__ unsigned s_warp[kPlanWarps];
  __shared__ unsigned s_total; // this CTA's count, read by the others
  __shared__ int s_long;       // a sequence would pass its row of the table
  __shared__ unsigned long long s_sum;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster.block_rank(), ctas = cluster.num_blocks();
  const int B = a.p.B, pages = a.p.num_pages, cap = a.p.max_pages << a.shift;
  if (tid == 0) s_long = 0, s_sum = 0;
  pdl_wait();
  // ---- the free (compact: live) pages of this warp's share of the pool: four adjacent ones a lane and
  // step, 128 a warp; the first eight steps' as a bit mask
  const int share = ((pages + ctas * kPlanWarps - 1) / (ctas * kPlanWarps) + 127) / 128 * 128;
  const long long begin = static_cast<long long>(rank * kPlanWarps + warp) * share;
  const int lo = static_cast<int>(min(begin, static_cast<long long>(pages)));
  const int hi = static_cast<int>(min(begin + share, static_cast<long long>(pages)));
  auto look = [&](int i) -> unsigned { // bits for pages i .. i + 3 (i a multiple of 4)
    if (i >= hi) return 0u;
    int r[4] = {1, 1, 1, 1};
    unsigned valid = 15u;
    if (i + 4 <= pages) {
      const int4 v = *reinterpret_cast<const int4 *>(a.p.refs + i);
      r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else {
      valid = (1u << (pages - i)) - 1u;
      for (int e = 0; i + e < pages; ++e) r[e] = a.p.refs[i + e];
    }
    const unsigned zero = (r[0] == 0) | (r[1] == 0) << 1 | (r[2] == 0) << 2 | (r[3] == 0) << 3;
    return (MODE == kCompact ? ~zero : zero) & valid;
  };
  unsigned held = 0; // the first eight looks
  unsigned cnt = 0;
  auto count = [&]() {
    held = cnt = 0;
#pragma unroll 1
    for (int i = lo + lane * 4, n = 0; i < hi; i += 128, ++n) {
      const unsigned m = look(i);
      if (n < 8) held |= m << (4 * n);
      cnt += __popc(m);
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
  };
  count();
  // ---- what each sequence needs (every CTA computes all of it)
  unsigned wanted = 0;
  if constexpr (MODE != kCompact) {
    const ForkWs f(a.ws, B);
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    auto need_of = [&](int b, int &had) -> unsigned {
      if constexpr (MODE == kExtend) {
        const int len = max(a.p.lens[b], 0);
        const long long after = static_cast<long long>(len) + max(a.in[b], 0);
        had = len <= cap ? pages_for(len, a.shift) : 0;
        if (after > cap) {
          s_long = 1;
          return 0u;
        }
        return pages_for(static_cast<int>(after), a.shift) - had;
      } else {
        const int par = a.in[b];
        const bool valid = static_cast<unsigned>(par) < static_cast<unsigned>(B) && par != b;
        const int len = valid ? min(max(a.p.lens[par], 0), cap) : 0;
        if (rank == 0) f.parent[b] = valid ? par : -1, f.len[b] = len, f.fresh[b] = -1;
        return (len & ((1 << a.shift) - 1)) != 0;
      }
    };
    unsigned sum = 0; // at most 4 * 2^26
    int had = 0;
    bool behind = false; // a sequence holds pages behind its length
#pragma unroll 1
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      sum += need_of(b, had);
      if constexpr (MODE == kExtend)
        behind |= had < a.p.max_pages && a.p.lens[b] <= cap &&
                  is_page(a.p, a.p.block_table[static_cast<long long>(b) * a.p.max_pages + had]);
    }
    if constexpr (MODE == kExtend) {
      // The caller lowered a length (every CTA sees it): the pages behind go back, and the counts are taken anew.
      if (__syncthreads_or(behind)) {
        if (ctas > 1) cluster.sync(); // every CTA has looked
        if (rank == 0)
#pragma unroll 1
          for (int b = warp; b < B; b += kPlanWarps)
            if (a.p.lens[b] <= cap) give_back(a.p, b, pages_for(max(a.p.lens[b], 0), a.shift), lane);
        if (ctas > 1) cluster.sync();
        else __syncthreads();
        count();
      }
    }
    unsigned run = block_scan(sum, s_warp, wanted);
    if (sum) atomicAdd(&s_sum, static_cast<unsigned long long>(sum)); // the scan may wrap; then the call fails
#pragma unroll 1
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      const unsigned need = need_of(b, had);
      s_pre[b] = run;
      if constexpr (MODE == kExtend) s_had[b] = had;
      run += need;
    }
  }
  unsigned all, before = block_scan(lane == 0 ? cnt : 0u, s_warp, all); // every lane of a warp: the warps before it
  before = __shfl_sync(0xffffffffu, before, 0);
  if (ctas > 1) {
    if (tid == 0) s_total = all;
    cluster.sync(); // totals are visible; every CTA has read lens and its part of refs
    all = 0;
    for (int r = 0; r < ctas; ++r) {
      const unsigned t = *cluster.map_shared_rank(&s_total, r);
      if (r < rank) before += t;
      all += t;
    }
    cluster.sync(); // nobody leaves while its total is being read
  } else {
    __syncthreads();
  }
  if constexpr (MODE != kCompact) {
    const int status = s_long ? 2 : s_sum > static_cast<unsigned long long>(all) ? 1 : 0;
    if (rank == 0 && tid == 0) {
      *a.status = status;
      if constexpr (MODE == kFork) ForkWs(a.ws, B).state[0] = status;
    }
    if (status != 0) {
      if (MODE == kExtend && rank == 0 && a.granted) // every CTA has read `in`
#pragma unroll 1
        for (int b = tid; b < B; b += kPlanThreads) a.granted[b] = 0;
      return;
    }
  } else if (rank == 0 && tid == 0) {
    *a.live = static_cast<int>(all);
    if (static_cast<int>(all) == pages) *CompactWs(a.ws, pages).moves = 0;
  }
  // ---- hand out the ranks
#pragma unroll 1
  for (int i0 = lo, n = 0; i0 < hi; i0 += 128, ++n) {
    if (MODE != kCompact && before >= wanted) break;
    const int i = i0 + lane * 4;
    const unsigned hit = n < 8 ? held >> (4 * n) & 15u : look(i);
    unsigned incl = __popc(hit);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    unsigned k = before + incl - __popc(hit); // free (live) pages before this one
    before += __shfl_sync(0xffffffffu, incl, 31);
    if constexpr (MODE == kCompact) {
      const CompactWs c(a.ws, pages);
      const int live = static_cast<int>(all);
#pragma unroll 1
      for (int page = i; page < min(i + 4, hi); ++page) {
        const bool is = hit >> (page - i) & 1u;
        if (page == live) *c.moves = live - static_cast<int>(k);
        if (page < live) {
          if (!is) c.hole[page - k] = page;
        } else {
          const int m = live - 1 - static_cast<int>(k); // live pages above this one
          if (is) c.src[m] = page;
          c.move_of[page] = is ? m : -1;
        }
        k += is;
      }
    } else {
#pragma unroll 1
      for (unsigned left = hit; left && k < wanted; left &= left - 1, ++k) {
        const int page = i + __ffs(left) - 1;
        int b0 = 0, b1 = B; // the last sequence with s_pre <= k
#pragma unroll 1
        while (b1 - b0 > 1) {
          const int mid = (b0 + b1) >> 1;
          (s_pre[mid] <= k ? b0 : b1) = mid;
        }
        if constexpr (MODE == kExtend) {
          const unsigned j = s_had[b0] + (k - s_pre[b0]); // within the row, unless lens changed meanwhile
          if (j < static_cast<unsigned>(a.p.max_pages)) a.p.block_table[static_cast<long long>(b0) * a.p.max_pages + j] = page;
        } else {
          ForkWs(a.ws, B).fresh[b0] = page;
        }
        a.p.refs[page] = 1;
      }
    }
  }
  if constexpr (MODE == kFork) {
    if (a.rows) {
      __syncthreads(); // parents, lengths and fresh pages are there
      const ForkWs f(a.ws, B);
#pragma unroll 1
      for (int b = warp; b < B; b += kPlanWarps) gather_row(a.p, a.shift, f, b, lane, 32);
      __syncthreads(); // every row has been read
#pragma unroll 1
      for (int b = warp; b < B; b += kPlanWarps) apply_row(a.p, a.shift, f, b, lane, 32);
    }
  }
  if (MODE == kExtend && rank == 0) { // every CTA has read lens (first cluster barrier)
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads) {
      const int add = max(a.in[b], 0);
      a.p.lens[b] = max(a.p.lens[b], 0) + add;
      if (a.granted) a.granted[b] = add;
    }
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
__global__ void __launch_bounds__(256) fork_rows_kernel(const tq_page_pool p, int shift, void *ws) {
  pdl_wait();
  const ForkWs f(ws, p.B);
  if (f.state[0] != 0) return;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y)
    gather_row(p, shift, f, b, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// Blocks of y = 0 write the table, lengths and counts; those of y = 1 (first: 0) copy the partial pages.
template <int N>
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const tq_page_pool p, int shift, int first,
                                                                  const __grid_constant__ Arrays<N> ar, void *ws) {
  pdl_wait();
  const ForkWs f(ws, p.B);
  if (f.state[0] != 0) return;
  if (static_cast<int>(blockIdx.y) + first == 0) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) apply_row(p, shift, f, b, threadIdx.x, kCopyThreads);
    return;
  }
  for (long long w = blockIdx.x; w < static_cast<long long>(p.B) * ar.units; w += gridDim.x) {
    const int b = static_cast<int>(w / ar.units);
    const int fresh = f.fresh[b];
    if (fresh < 0) continue;
    const int src = f.rows[static_cast<long long>(b) * p.max_pages + (f.len[b] >> shift)];
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

int shift_of(const tq_page_pool &p) {
  int n = 0;
  while ((1 << n) < p.page_size) ++n;
  return n;
}

cudaError_t launch_plan(void (*kernel)(PlanArgs), cudaStream_t s, const PlanArgs &a) {
  const unsigned ctas = a.p.num_pages <= kSmallPool ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
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

cudaError_t launch_pages_extend(const tq_page_pool &p, const int *need, int *granted, int *status, cudaStream_t s) {
  return launch_plan(plan_kernel<kExtend>, s, PlanArgs{p, shift_of(p), need, status, granted, nullptr, nullptr, false});
}

cudaError_t launch_pages_fork(const tq_page_pool &p, const tq_page_array *arrays, int n_arrays,
                              const int *parent_of, int *status, void *ws, int sm_count, cudaStream_t s) {
  // One CTA also gathers and writes a small table's rows and saves a launch, about 2 us of host time. GPU
  // time of a fork so, and over the whole GPU (in brackets without arrays to copy): 8 x 16 entries 9.3
  // against 9.8 (7.4, 9.8) us, 32 x 64 11.9 against 12.1 (9.5, 12.3), 64 x 64 14.2 against 13.5 (11.6, 13.4),
  // 64 x 128 15.7 against 13.7 (13.0, 13.5). A row is one warp's: few long rows, 4 x 1024, take 19 against 11.
  const bool rows = p.num_pages <= kSmallPool && static_cast<long long>(p.B) * p.max_pages <= kSmallTable;
  cudaError_t e = launch_plan(plan_kernel<kFork>, s, PlanArgs{p, shift_of(p), parent_of, status, nullptr, nullptr, ws, rows});
  if (e != cudaSuccess || (rows && n_arrays == 0)) return e;
  if (!rows) {
    e = launch_pdl(fork_rows_kernel, row_grid(p), dim3(256), 0, s, p, shift_of(p), ws);
    if (e != cudaSuccess) return e;
  }
  return with_arrays(arrays, n_arrays, [&](const auto &ar) {
    using A = std::decay_t<decltype(ar)>;
    constexpr int N = sizeof(A) > sizeof(Arrays<kFewArrays>) ? kMaxPageArrays : kFewArrays;
    const dim3 grid(sm_count * 8, (n_arrays > 0) + !rows);
    return launch_pdl(fork_apply_kernel<N>, grid, dim3(kCopyThreads), 0, s, p, shift_of(p), static_cast<int>(rows), ar, ws);
  });
}

cudaError_t launch_pages_free(const tq_page_pool &p, const int *leaving, cudaStream_t s) {
  return launch_pdl(free_kernel, row_grid(p), dim3(256), 0, s, p, leaving);
}

cudaError_t launch_pages_compact(const tq_page_pool &p, const tq_page_array *arrays, int n_arrays, int *live,
                                 void *ws, int sm_count, cudaStream_t s) {
  cudaError_t e = launch_plan(plan_kernel<kCompact>, s, PlanArgs{p, shift_of(p), nullptr, nullptr, nullptr, live, ws, false});
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
