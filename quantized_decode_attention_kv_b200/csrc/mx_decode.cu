// Attention of one or a few queries of every sequence over the microscaled 4-bit paged cache.
//
// o = sum_j softmax_j(scale q.k_j) v_j with k_j, v_j = E2M1 * S * g. Everything is transposed so
// that the tensor-core tile's 16 rows are tokens (scores) or head elements (values) and its 8
// columns are query rows (query, head of the KV head's group): one decode query of a group of 8
// wastes nothing.
//   scores  S^T[16 tokens x 8]  = K[16 x D] . q^T[D x 8]      (A: codes turned into fp16 registers)
//   values  O^T[D x 8]         += V^T[D x 16] . P^T[16 x 8]   (A: codes of token pairs)
// E2M1 * E4M3 has 6 significant bits and spans 2^-10..2688, so fp16 operands are exact; queries
// are fp16 after a power-of-two scaling of each row (exact for fp16; for bf16 exact down to
// 2^-32 of the row's largest element). Products and sums are fp32. P is held in fp16 with the
// row's reference moved by 2^11..2^15, so that weights down to 2^-25 of the largest keep 11 bits;
// the row sums come from the same rounded weights (an MMA with ones), which cancels most of that
// rounding.
//
// The softmax reference of a row moves only when a score passes it by 2^15 (a vote in the warp);
// the frequent path has no cross-lane reduction.
//
// Work: the (sequence, KV head, row block, 16-token tile) space is flattened and divided evenly
// over the CTAs on the device, from the lengths in device memory, so a captured graph follows
// lengths that change and a ragged batch stays balanced. A CTA's warps share each stretch and
// merge in shared memory; a unit cut by a CTA boundary leaves partials in the workspace for the
// combine kernel.
#include <cfloat>

#include "mma_ops.cuh"
#include "mx.cuh"

namespace tq {
namespace {

using namespace mx;
using namespace mma_ops;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kRefDrop = 11.0f;  // the reference sits 2^11 below the largest score seen ...
constexpr float kRefSlack = 15.0f; // ... and follows when a weight would pass 2^15 (fp16 ends at 2^16)
constexpr float kRefEmpty = -FLT_MAX;
constexpr int kMinTiles = 8; // tiles a CTA gets at least: one for each warp

struct Kernel {
  MxCacheArgs c;
  const uint16_t *q;
  const int *lens, *counts;
  void *out;
  float *part;   // [2 * ctas][8 NT][D + 2]: output sums, then reference and weight sum
  int4 *desc;    // [ctas]: {sequence, head, row block, number of CTAs} of the unit cut at its end
  int Hq, G, Lq, row_blocks, bf16, out_dtype;
  float scale, klog; // softmax scale; log2(e) * key scale (apart: their product may not fit where a row's does)
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ int tiles_of(const Kernel &k, int b) {
  if (clamp_count(k.counts, b, k.Lq) == 0) return 0;
  const int cap = k.c.maxp << k.c.pshift;
  return (min(max(__ldg(k.lens + b), 0), cap) + 15) >> 4;
}

__device__ __forceinline__ void store_out(const Kernel &k, long long i, float a, float b) {
  if (k.out_dtype == TQ_F32) {
    *reinterpret_cast<float2 *>(static_cast<float *>(k.out) + i) = make_float2(a, b);
  } else if (k.out_dtype == TQ_BF16) {
    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(k.out) + i) = __floats2bfloat162_rn(a, b);
  } else {
    *reinterpret_cast<__half2 *>(static_cast<__half *>(k.out) + i) = __floats2half2_rn(a, b);
  }
}

// Position limits of a row of a unit: row r is query r / G, head r % G of the group; it sees
// positions below limit(r) (0: none).
struct Rows {
  int count, first, seen; // queries of the sequence, position of query 0, cached positions
  __device__ __forceinline__ int limit(int query) const {
    return query < count ? min(max(first + query + 1, 0), seen) : 0;
  }
};
__device__ __forceinline__ Rows rows_of(const Kernel &k, int b) {
  Rows r;
  const int len = __ldg(k.lens + b), cap = k.c.maxp << k.c.pshift;
  r.count = clamp_count(k.counts, b, k.Lq);
  r.first = len - r.count;
  r.seen = min(max(len, 0), cap);
  return r;
}

// Codes and scale bytes of one 16-token tile, as a lane holds them: rows g and g + 8 of the keys
// (D/4 elements each, from element tig * D/4), tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9 of
// the values (D/8 elements each, from element g * D/8).
template <int D>
struct Tile {
  uint32_t k[2][D / 32], v[4][D / 64];
  uint32_t ks[2], vs[4];
  bool mapped;
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
  }
}

template <int N> // N scale bytes (1, 2 or 4)
__device__ __forceinline__ uint32_t load_scales(const uint8_t *p) {
  if constexpr (N == 1) return __ldg(p);
  else if constexpr (N == 2) return __ldg(reinterpret_cast<const uint16_t *>(p));
  else return __ldg(reinterpret_cast<const uint32_t *>(p));
}

// The block-table row of a sequence, 32 entries at a time across the warp's lanes.
struct TableWindow {
  const int *row;
  int maxp, base, entry;
  __device__ __forceinline__ void start(const int *r, int n) {
    row = r;
    maxp = n;
    base = -1;
    entry = -1;
  }
  __device__ __forceinline__ int page(int p, int lane) { // p: the same in every lane
    if ((p & ~31) != base) {
      base = p & ~31;
      entry = base + lane < maxp ? __ldg(row + base + lane) : -1;
    }
    return __shfl_sync(0xffffffffu, entry, p & 31);
  }
};

template <int D>
__device__ __forceinline__ void load_tile(const Kernel &k, TableWindow &win, int h, int tile, int lane, Tile<D> &t) {
  const int g = lane >> 2, tig = lane & 3, pos = tile << 4;
  const int page = win.page(pos >> k.c.pshift, lane);
  t.mapped = page >= 0 && page < k.c.num_pages;
  // records < 2^32 (the host checks), so the record index is one 32-bit word
  const uint32_t rec = (((t.mapped ? page : 0) * static_cast<uint32_t>(k.c.Hkv) + h) << k.c.pshift) +
                       (pos & ((1 << k.c.pshift) - 1));
  const uint8_t *kc = k.c.codes[0] + static_cast<size_t>(rec) * (D / 2) + g * (D / 2) + tig * (D / 8);
  const uint8_t *ks = k.c.scales[0] + static_cast<size_t>(rec) * (D / 16) + g * (D / 16) + tig * (D / 64);
  const uint8_t *vc = k.c.codes[1] + static_cast<size_t>(rec) * (D / 2) + tig * D + g * (D / 16);
  const uint8_t *vs = k.c.scales[1] + static_cast<size_t>(rec) * (D / 16) + tig * (D / 8) + g * D / 128;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    load_words(kc + r * 8 * (D / 2), t.k[r]);
    t.ks[r] = load_scales<D / 64>(ks + r * 8 * (D / 16));
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int row = (s >> 1) * 8 + (s & 1);
    load_words(vc + row * (D / 2), t.v[s]);
    t.vs[s] = load_scales<(D == 256 ? 2 : 1)>(vs + row * (D / 16));
  }
}

// One warp's running state over its tiles.
template <int D, int NT>
struct Acc {
  float o[NT][D / 16][4];
  float l[NT][4];   // weight sums of columns 2 tig, 2 tig + 1 (rows of the ones tile: all equal)
  float ref[NT][2]; // reference of those columns, log2 units
};

// P.V of one tile: p = the weight fragments, token pairs' scales in vs. kOwn: only the columns with
// their bit in `own` (bit 2 n + c: column 2 tig + c of tile n) take the products.
template <int D, int NT, bool kOwn>
__device__ __forceinline__ void add_values(const Tile<D> &t, const uint32_t (&vs)[4], const uint32_t (&p)[NT][2],
                                           Acc<D, NT> &acc, unsigned own = 0) {
  constexpr int kS = D == 256 ? 2 : 1;
  uint32_t sc[2][kS]; // scale pairs (token, token + 1)
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int b = 0; b < kS; ++b)
      sc[u][b] = e4m3_to_h2(prmt(vs[2 * u], vs[2 * u + 1], b == 0 ? 0x4440u : 0x5551u));
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    uint32_t even[2][4], odd[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t a = t.v[2 * u][w], b = t.v[2 * u + 1][w];
      e2m1_to_h2((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), even[u]);
      e2m1_to_h2(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), odd[u]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0 = hmul2(even[0][j], sc[0][w / 2]), a1 = hmul2(odd[0][j], sc[0][w / 2]);
      const uint32_t a2 = hmul2(even[1][j], sc[1][w / 2]), a3 = hmul2(odd[1][j], sc[1][w / 2]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (!kOwn) {
          mma16816(acc.o[n][4 * w + j], a0, a1, a2, a3, p[n][0], p[n][1]);
        } else {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(c, a0, a1, a2, a3, p[n][0], p[n][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (own >> (2 * n + (e & 1)) & 1u) acc.o[n][4 * w + j][e] += c[e];
        }
      }
    }
  }
}

// One tile. kMasked: some row of the block does not see every token of the tile (or its page is
// unmapped); `limit` then holds the columns' position limits.
template <int D, int NT, bool kMasked>
__device__ __forceinline__ void do_tile(const Tile<D> &t, const uint32_t (&q)[NT][D / 8], const float (&mul)[NT][2],
                                        const int (&limit)[NT][2], const Rows &rows, int row0, int G, int pos,
                                        int lane, Acc<D, NT> &acc) {
  const int g = lane >> 2, tig = lane & 3;
  float s[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    uint32_t a[4], b[4];
    e2m1_to_h2(t.k[0][w], a);
    e2m1_to_h2(t.k[1][w], b);
    // the scale of this word's block, in both halves
    const uint32_t sel = (w / 2) * 0x11u;
    const uint32_t sa = e4m3_to_h2(prmt(t.ks[0], 0u, sel | 0x4400u)), sb = e4m3_to_h2(prmt(t.ks[1], 0u, sel | 0x4400u));
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = hmul2(a[j], sa), b[j] = hmul2(b[j], sb);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma16816(s[n], a[0], b[0], a[1], b[1], q[n][4 * w], q[n][4 * w + 1]);
      mma16816(s[n], a[2], b[2], a[3], b[3], q[n][4 * w + 2], q[n][4 * w + 3]);
    }
  }
  float x[NT][4]; // logits (log2 units) less the column's reference
  bool move = false;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[n][e] *= mul[n][e & 1];
      if (kMasked && (pos + g + (e >> 1) * 8 >= limit[n][e & 1] || !t.mapped)) s[n][e] = -INFINITY;
      x[n][e] = s[n][e] - acc.ref[n][e & 1];
      move |= x[n][e] > kRefSlack;
    }
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = fmaxf(acc.ref[n][c], top - kRefDrop), f = softmax_exp2(acc.ref[n][c] - ref);
        acc.ref[n][c] = ref;
        x[n][c] = s[n][c] - ref;
        x[n][c + 2] = s[n][c + 2] - ref;
        acc.l[n][c] *= f;
        acc.l[n][c + 2] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc.o[n][i][c] *= f, acc.o[n][i][c + 2] *= f;
      }
    }
  }
  uint32_t p[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    p[n][0] = transpose8x8(pack_h2(softmax_exp2(x[n][0]), softmax_exp2(x[n][1])));
    p[n][1] = transpose8x8(pack_h2(softmax_exp2(x[n][2]), softmax_exp2(x[n][3])));
    mma16816(acc.l[n], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, p[n][0], p[n][1]);
  }
  if constexpr (!kMasked) {
    add_values<D, NT, false>(t, t.vs, p, acc);
  } else {
    // 0 * NaN is NaN: a token that a row does not see must not reach it through its scale either.
    // Tokens that no row sees get scale 0. A NaN scale among the rest of a masked tile is rare;
    // then each query of the block takes its own pass with only its own tokens and columns.
    uint32_t vs[4];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vs[i] = pos + 2 * tig + (i >> 1) * 8 + (i & 1) < rows.seen && t.mapped ? t.vs[i] : 0u;
      nan |= (vs[i] & 0x7Fu) == 0x7Fu || (vs[i] & 0x7F00u) == 0x7F00u;
    }
    if (!__any_sync(0xffffffffu, nan)) {
      add_values<D, NT, false>(t, vs, p, acc);
    } else {
      const int last = min((row0 + 8 * NT - 1) / G, rows.count - 1);
      for (int query = row0 / G; query <= last; ++query) {
        const int lim = rows.limit(query);
        uint32_t pq[NT][2], vq[4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool mine = (row0 + 8 * n + g) / G == query; // a fragment's column is row g
          pq[n][0] = mine ? p[n][0] : 0u;
          pq[n][1] = mine ? p[n][1] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) vq[i] = pos + 2 * tig + (i >> 1) * 8 + (i & 1) < lim ? vs[i] : 0u;
        // columns of other queries still meet this pass's NaN scales, with weight 0
        unsigned own = 0;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
          own |= static_cast<unsigned>((row0 + 8 * (i >> 1) + 2 * tig + (i & 1)) / G == query) << i;
        add_values<D, NT, true>(t, vq, pq, acc, own);
      }
    }
  }
}

template <int D, int NT>
constexpr int smem_bytes() {
  return kWarps * 8 * NT * (D + 4) * 4 + kWarps * 8 * NT * 2 * 4;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, D == 256 || NT > 1 ? 1 : 2) mx_decode_kernel(const Kernel k) {
  constexpr int R = 8 * NT;   // rows of a block
  constexpr int kP = D + 4;   // padded row of the merge buffer
  extern __shared__ float sm[];
  float *so = sm, *sr = sm + kWarps * R * kP; // [warp][R][kP]; [warp][R]{reference, sum}
  __shared__ long long s_scan[kWarps];
  __shared__ long long s_start;
  __shared__ int s_b0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  pdl_wait();
  // ---- this CTA's stretch of the flattened tile space
  const int B = k.c.B, per = (B + kThreads - 1) / kThreads;
  const long long heads = static_cast<long long>(k.c.Hkv) * k.row_blocks;
  long long mine = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < B) mine += tiles_of(k, tid * per + i);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  total *= heads;
  const long long n = min(static_cast<long long>(gridDim.x), max(total / kMinTiles, 1ll));
  const int cta = blockIdx.x;
  const long long lo = cta < n ? total * cta / n : total, hi = cta < n ? total * (cta + 1) / n : total;
  long long at = (before + incl - mine) * heads;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= B) break;
    const long long len = tiles_of(k, b) * heads;
    if (lo >= at && lo < at + len) s_b0 = b, s_start = at;
    at += len;
  }
  // sequences without tiles have only empty rows
  for (int b = cta; b < B; b += gridDim.x) {
    if (tiles_of(k, b)) continue;
    const long long base = static_cast<long long>(b) * k.Lq * k.Hq * D;
    for (long long i = 2 * tid; i < static_cast<long long>(k.Lq) * k.Hq * D; i += 2 * kThreads)
      store_out(k, base + i, 0.0f, 0.0f);
  }
  __syncthreads();
  if (lo >= hi) {
    if (tid == 0) k.desc[cta] = make_int4(0, 0, 0, 0);
    return;
  }
  int b = s_b0;
  long long start = s_start, cur = lo; // first tile of sequence b, and of this stretch
  int4 desc = make_int4(0, 0, 0, 0);
  while (cur < hi) {
    int nt_b = tiles_of(k, b);
    while (cur >= start + nt_b * heads) { // next sequence that has tiles
      start += nt_b * heads;
      nt_b = tiles_of(k, ++b);
    }
    const long long unit = (cur - start) / nt_b, unit0 = start + unit * nt_b;
    const int h = static_cast<int>(unit / k.row_blocks), rb = static_cast<int>(unit - static_cast<long long>(h) * k.row_blocks);
    const int t0 = static_cast<int>(cur - unit0), t1 = static_cast<int>(min(static_cast<long long>(nt_b), hi - unit0));
    const Rows rows = rows_of(k, b);
    const int row0 = rb * R;
    // ---- queries: row g of each column tile, scaled by a power of two into fp16
    uint32_t q[NT][D / 8];
    float mul[NT][2];
    int limit[NT][2];
    int full = rows.seen; // every row of the block sees the positions below
#pragma unroll
    for (int n_ = 0; n_ < NT; ++n_) {
      const int row = row0 + 8 * n_ + g, query = row / k.G;
      float x[D / 4];
      float top = 0.0f;
      if (query < rows.count) {
        const uint16_t *src = k.q + ((static_cast<long long>(b) * k.Lq + query) * k.Hq + h * k.G + row % k.G) * D + tig * (D / 4);
        if (k.bf16) load_vec<D / 4>(src, TQ_BF16, 0, x);
        else load_vec<D / 4>(src, TQ_F16, 0, x);
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent that brings the largest element to 2^14..2^15; a row of zeros, infinities or NaN
      // keeps its values
      const int e = top > 0.0f && top < INFINITY ? 14 - ilogbf(top) : 0;
      const float f1 = ldexpf(1.0f, e / 2), f2_ = ldexpf(1.0f, e - e / 2);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) q[n_][i] = pack_h2(x[2 * i] * f1 * f2_, x[2 * i + 1] * f1 * f2_);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ec = __shfl_sync(0xffffffffu, e, (2 * tig + c) * 4);
        mul[n_][c] = ldexpf(k.scale, -ec) * k.klog;
        const int qc = (row0 + 8 * n_ + 2 * tig + c) / k.G;
        limit[n_][c] = qc < rows.count ? rows.limit(qc) : rows.seen;
      }
    }
    if (row0 / k.G < rows.count) full = rows.limit(row0 / k.G);
    // ---- the warp's tiles
    Acc<D, NT> acc;
#pragma unroll
    for (int n_ = 0; n_ < NT; ++n_) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.o[n_][i][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc.l[n_][e] = 0.0f;
      acc.ref[n_][0] = acc.ref[n_][1] = kRefEmpty;
    }
    const int share = (t1 - t0 + kWarps - 1) / kWarps;
    const int w0 = min(t0 + warp * share, t1), w1 = min(w0 + share, t1);
    if (w0 < w1) {
      TableWindow win;
      win.start(k.c.bt + static_cast<long long>(b) * k.c.maxp, k.c.maxp);
      Tile<D> cur_t, next_t;
      load_tile<D>(k, win, h, w0, lane, cur_t);
      for (int tile = w0; tile < w1; ++tile) {
        if (tile + 1 < w1) load_tile<D>(k, win, h, tile + 1, lane, next_t);
        const int pos = tile << 4;
        if (pos + 16 <= full && cur_t.mapped)
          do_tile<D, NT, false>(cur_t, q, mul, limit, rows, row0, k.G, pos, lane, acc);
        else
          do_tile<D, NT, true>(cur_t, q, mul, limit, rows, row0, k.G, pos, lane, acc);
        cur_t = next_t;
      }
    }
    // ---- merge the warps
    __syncthreads(); // the buffer's readers of the stretch before are done
#pragma unroll
    for (int n_ = 0; n_ < NT; ++n_)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n_ + 2 * tig + c;
        if (g == 0) {
          sr[(warp * R + r) * 2] = acc.ref[n_][c];
          sr[(warp * R + r) * 2 + 1] = acc.l[n_][c];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2 *>(so + (warp * R + r) * kP + g * (D / 8) + 2 * i) =
              make_float2(acc.o[n_][i][c], acc.o[n_][i][c + 2]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt_b;
    float *slot = k.part + static_cast<long long>(2 * cta + (t0 == 0 ? 1 : 0)) * R * (D + 2);
    for (int i = tid; i < R * (D / 2); i += kThreads) {
      const int r = i / (D / 2), d = 2 * (i - r * (D / 2));
      float ref = kRefEmpty, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, sr[(w * R + r) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = softmax_exp2(sr[(w * R + r) * 2] - ref);
        const float2 v = *reinterpret_cast<const float2 *>(so + (w * R + r) * kP + d);
        l += f * sr[(w * R + r) * 2 + 1];
        o0 += f * v.x;
        o1 += f * v.y;
      }
      if (whole) {
        const int query = (row0 + r) / k.G;
        if (query < k.Lq) {
          // the largest weight is 2^11 or more: a sum of 0 means that every position was unmapped
          const bool some = rows.limit(query) > 0 && l != 0.0f;
          const float inv = k.c.g[1] / l;
          store_out(k, ((static_cast<long long>(b) * k.Lq + query) * k.Hq + h * k.G + (row0 + r) % k.G) * D + d,
                    some ? o0 * inv : 0.0f, some ? o1 * inv : 0.0f);
        }
      } else {
        *reinterpret_cast<float2 *>(slot + r * D + d) = make_float2(o0, o1);
        if (d == 0) slot[R * D + 2 * r] = ref, slot[R * D + 2 * r + 1] = l;
      }
    }
    if (!whole && t0 == 0) { // the unit goes on in the CTAs behind: this one describes it
      const long long end = unit0 + nt_b;
      const int last = static_cast<int>((end * n - 1) / total);
      desc = make_int4(b, h, rb, last - cta + 1);
    }
    cur = unit0 + t1;
  }
  if (tid == 0) k.desc[cta] = desc;
}

// Joins the partials of a unit that several CTAs share: parts 0 (slot 1 of its first CTA) and
// 1.. (slot 0 of the CTAs behind it). One CTA for each boundary; most return at once.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) mx_combine_kernel(const Kernel k) {
  constexpr int R = 8 * NT;
  pdl_wait();
  const int cta = blockIdx.x;
  const int4 d = k.desc[cta];
  if (d.w == 0) return;
  const int b = d.x, h = d.y, row0 = d.z * R, parts = d.w;
  const Rows rows = rows_of(k, b);
  const long long stride = static_cast<long long>(R) * (D + 2);
  const float *first = k.part + (2ll * cta + 1) * stride, *rest = k.part + 2ll * (cta + 1) * stride;
  for (int i = threadIdx.x; i < R * (D / 2); i += kThreads) {
    const int r = i / (D / 2), e = 2 * (i - r * (D / 2));
    const int query = (row0 + r) / k.G;
    if (query >= k.Lq) continue;
    float o0 = 0.0f, o1 = 0.0f, l = 0.0f;
    const bool some = rows.limit(query) > 0;
    if (some) {
      float ref = first[R * D + 2 * r];
      for (int p = 0; p + 1 < parts; ++p) ref = fmaxf(ref, rest[2 * p * stride + R * D + 2 * r]);
#pragma unroll 4
      for (int p = 0; p < parts; ++p) {
        const float *s = p == 0 ? first : rest + 2 * (p - 1) * stride;
        const float f = softmax_exp2(s[R * D + 2 * r] - ref);
        const float2 v = *reinterpret_cast<const float2 *>(s + r * D + e);
        l += f * s[R * D + 2 * r + 1];
        o0 += f * v.x;
        o1 += f * v.y;
      }
      const float inv = l != 0.0f ? k.c.g[1] / l : 0.0f; // as above
      o0 *= inv;
      o1 *= inv;
    }
    store_out(k, ((static_cast<long long>(b) * k.Lq + query) * k.Hq + h * k.G + (row0 + r) % k.G) * D + e, o0, o1);
  }
}

template <int D, int NT>
cudaError_t run(const Kernel &k, const MxPlan &p, cudaStream_t s) {
  constexpr int smem = smem_bytes<D, NT>();
  cudaError_t e = cudaFuncSetAttribute(mx_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(mx_decode_kernel<D, NT>, dim3(p.ctas), dim3(kThreads), smem, s, k);
  if (e != cudaSuccess) return e;
  return launch_pdl(mx_combine_kernel<D, NT>, dim3(p.ctas), dim3(kThreads), 0, s, k);
}

} // namespace

MxPlan plan_mx_decode(int Hkv, int d, int Hq, int Lq, int sm_count) {
  MxPlan p;
  const int rows = Lq * (Hq / Hkv);
  p.nt = d < 256 && rows > 8 ? 2 : 1;
  p.row_blocks = (rows + 8 * p.nt - 1) / (8 * p.nt);
  p.ctas = sm_count * (d == 256 || p.nt > 1 ? 1 : 2);
  // partials of one launch: 2 ctas x 8 nt rows, the same for both tile counts; one descriptor per
  // CTA, at most two CTAs an SM. One size serves every number of queries and heads.
  p.ws_bytes = static_cast<size_t>(4) * sm_count * 8 * (d + 2) * sizeof(float) + 2 * sm_count * sizeof(int4);
  return p;
}

cudaError_t launch_mx_decode(const MxDecodeArgs &a, cudaStream_t s) {
  Kernel k;
  k.c = a.c;
  k.q = static_cast<const uint16_t *>(a.q);
  k.lens = a.lens;
  k.counts = a.counts;
  k.out = a.out;
  k.desc = static_cast<int4 *>(a.ws);
  k.part = reinterpret_cast<float *>(k.desc + a.plan.ctas);
  k.Hq = a.Hq;
  k.G = a.Hq / a.c.Hkv;
  k.Lq = a.Lq;
  k.row_blocks = a.plan.row_blocks;
  k.bf16 = a.dtype == TQ_BF16;
  k.out_dtype = a.out_dtype;
  k.scale = a.scale;
  k.klog = 1.4426950408889634f * a.c.g[0];
  if (a.c.d == 64) return a.plan.nt == 1 ? run<64, 1>(k, a.plan, s) : run<64, 2>(k, a.plan, s);
  if (a.c.d == 128) return a.plan.nt == 1 ? run<128, 1>(k, a.plan, s) : run<128, 2>(k, a.plan, s);
  return run<256, 1>(k, a.plan, s);
}

} // namespace tq
