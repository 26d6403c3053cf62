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
// Work: the space of 32-token tiles of all (sequence, KV head, row block) units is flattened and
// divided evenly over all warps of the grid on the device, from the lengths in device memory, so a
// captured graph follows lengths that change and a ragged batch stays balanced. A unit counts
// kUnitCost tiles more than it has (queries, page table, output). Each warp copies its own tiles
// with cp.async into a ring of its own, ahead across units, and waits for no other warp until its
// stretch is done. Units within a stretch are finished by their warp; the others leave partials in
// shared memory, joined by the CTA, and those cut by a CTA boundary in the workspace, joined by the
// combine kernel. (With a CTA's warps sharing each unit, meeting at its end, a ragged batch of 32 took
// 155 us; this way 25 us. Joining in the CTA that arrives last, in place of the combine kernel, saved
// 2.4 us on the host and cost up to 9 us on the GPU, where one CTA had two long joins to do.)
//
// A sequence with fewer queries than the batch's widest (counts[b] < Lq) takes all row blocks all the same:
// those without a query of it cost as much as the others and end as zeros. (Drafts of 0 to 5 queries at 4
// query heads, blocks of 8 rows: 48% of the steps.)
//
// Bound: HBM by its bytes (144 a token and KV head at D = 128); in practice the latency of each warp's
// chain of instructions. 16 x 32K positions of 8 heads, D = 128, 4 query heads each: 604 MB in 134 us over
// rotating inputs (4.5 TB/s, 69% of the copy rate), 118 us in replays over one, where the copies alone
// take 99. 273 warp instructions for 16 tokens, of which 64 conversions, 64 scalings and 17 MMAs, fill 58% of
// the issue slots: registers leave a scheduler 3 warps, 1 of them ready on average, and they wait for fixed
// latencies and busy pipes (2.3 of 4.8 cycles an instruction), hardly for memory (0.1). Heads of 64: 64% with
// 4 warps. A step takes 32 tokens: with 16 it took 314 instructions and 126 us.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "mma_ops.cuh"
#include "mx.cuh"

namespace tq {
namespace {

using namespace mx;
using namespace mma_ops;

constexpr float kRefDrop = 11.0f;  // the reference sits 2^11 below the largest score seen ...
constexpr float kRefSlack = 15.0f; // ... and follows when a weight would pass 2^15 (fp16 ends at 2^16)
constexpr float kRefEmpty = -FLT_MAX;
// Weight sum of a row that has seen mapped positions, all with scores of -infinity: its softmax is NaN, where
// a row that has seen none (sum 0) gives zeros. It vanishes beside any weight of a finite score (the largest
// is 1 or more) and stays below kLostBelow in joins of any number of stretches.
constexpr float kLost = 0x1p-100f, kLostBelow = 0x1p-60f;
// Shapes of the grid: CTAs of an SM, tiles in a warp's ring. One column tile of D = 128 needs about 165
// registers: 12 warps an SM of 168 take 128 us for 16 x 32K positions, 16 warps of 128 spill (146 us).
// More column tiles keep their queries in shared memory (four queries of 8 x 9001 positions: 57 us with
// them in registers, 39 us).
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
template <int D, int NT>
struct Cfg {
  static constexpr int kCtas = D == 64 && NT == 1 ? 4 : D == 256 || (D == 128 && NT == 2) ? 2 : 3;
  static constexpr bool kQueriesInSmem = NT > 1;
  static constexpr int kStages = D == 256 ? 2 : 3; // what fits (D = 256, 8 warps: 16 x 16K positions, 604 MB, 113 us)
  static constexpr int kSixteen = 18 * D;            // bytes: 16 x (D/2 + D/16) of keys and of values
  static constexpr int kTile = kSub * kSixteen;
  static constexpr int kSlot = 8 * NT * (D + 2) * 4; // bytes of a partial: sums, then (reference, weight sum)
  static constexpr int kQueries = kQueriesInSmem ? 16 * D * NT : 0;
  static constexpr int kWarpBytes = kStages * kTile + kSlot + kQueries;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert(kCtas * (kSmem + 2048) <= 228 * 1024, "the CTAs of an SM are resident together");
  static constexpr int kHeadAt = kStages * kTile + kQueries; // of the slot for the stretch's first unit
  static_assert(kSlot <= kHeadAt && kTile % 16 == 0 && kSlot % 16 == 0, "the tail's partial reuses ring and queries");
};

struct Kernel {
  MxCacheArgs c;
  const uint16_t *q;
  const int *lens, *counts;
  void *out;
  float *part;   // [2 * ctas] partials (Cfg::kSlot)
  int4 *desc;    // [ctas]: {sequence, head, first row, number of CTAs} of the unit cut at its end
  int Hq, G, Lq, row_blocks, bf16, out_dtype;
  float inv_group;   // 1 / G
  float scale, klog; // softmax scale; log2(e) * key scale (apart: their product may not fit where a row's does)
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<uint32_t *>(&r);
}
// The low halves of a's bytes and the high halves of b's.
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Row r of a unit is query r / G, head r % G of the group. The quotient is at most 40 and G below
// 2^16, so the float product is off by less than the half step that separates it from a whole number.
__device__ __forceinline__ int query_of(const Kernel &k, int row) {
  return static_cast<int>((static_cast<float>(row) + 0.5f) * k.inv_group);
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

// Codes and scale bytes of one 16-token tile, as a lane holds them: rows g and g + 8 of the keys
// (D/4 elements each, from element tig * D/4), tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9 of
// the values (D/8 elements each, from element g * D/8).
template <int D>
struct Tile {
  uint32_t k[2][D / 32], v[4][D / 64];
  uint32_t ks[2], vs[4];
};

// A tile in a ring: key codes [16][D/2], value codes [16][D/2], key scales [16][D/16], value scales
// [16][D/16]. The eight 16-byte chunks of a 128-byte line of codes are permuted by the line (XOR), so
// that the lanes' reads (rows g by tig for keys, tokens 2 tig + i by g for values) meet no bank twice.
template <int D>
__device__ __forceinline__ int chunk_swizzle(int line) {
  return D == 64 ? 2 * (line & 1) : D == 128 ? 2 * (line & 3) : line & 7;
}
template <int D>
__device__ __forceinline__ int code_offset(int token, int byte) { // byte: of the token's record, < D/2
  const int at = token * (D / 2) + byte, line = at >> 7;
  return line * 128 + ((((at >> 4) & 7) ^ chunk_swizzle<D>(line)) << 4) + (at & 15);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int N> // 4-byte words
__device__ __forceinline__ void lds(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]) : "r"(a ^ (4 * i)));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a));
  }
}
template <int N> // 1, 2 or 4 bytes
__device__ __forceinline__ uint32_t lds_bytes(uint32_t a) {
  uint32_t w;
  if constexpr (N == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w) : "r"(a));
  else if constexpr (N == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(a));
  else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(a));
  return w;
}

// Where a lane reads in a tile: its keys (row g; row g + 8 is 4 D bytes on), values (tokens 2 tig
// and 2 tig + 1; those 8 on are 4 D bytes on) and scales. They go through a shuffle because the
// compiler would otherwise compute them anew for every tile to save registers.
template <int D>
struct Reads {
  uint32_t k, v[2], ks, vs;
  __device__ __forceinline__ explicit Reads(int lane) {
    const int g = lane >> 2, tig = lane & 3;
    k = code_offset<D>(g, tig * (D / 8));
    v[0] = 8 * D + code_offset<D>(2 * tig, g * (D / 16));
    v[1] = 8 * D + code_offset<D>(2 * tig + 1, g * (D / 16));
    ks = 16 * D + g * (D / 16) + tig * (D / 64);
    vs = 17 * D + 2 * tig * (D / 16) + (D == 64 ? g / 2 : D == 128 ? g : 2 * g);
    k = __shfl_sync(0xffffffffu, k, lane);
    v[0] = __shfl_sync(0xffffffffu, v[0], lane);
    v[1] = __shfl_sync(0xffffffffu, v[1], lane);
    ks = __shfl_sync(0xffffffffu, ks, lane);
    vs = __shfl_sync(0xffffffffu, vs, lane);
  }
};
template <int D>
__device__ __forceinline__ void read_keys(uint32_t sm, const Reads<D> &at, Tile<D> &t) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    // the swizzle of rows 8 apart is the same; a lane's 32 bytes of D = 256 are two chunks of one XOR
    lds(sm + at.k + r * 4 * D, t.k[r]);
    t.ks[r] = lds_bytes<D / 64>(sm + at.ks + r * (D / 2));
  }
}
template <int D>
__device__ __forceinline__ void read_values(uint32_t sm, const Reads<D> &at, Tile<D> &t) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    lds(sm + at.v[s & 1] + (s >> 1) * 4 * D, t.v[s]);
    t.vs[s] = lds_bytes<(D == 256 ? 2 : 1)>(sm + at.vs + ((s >> 1) * 8 + (s & 1)) * (D / 16));
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
      e2m1_to_h2(select_bits(a, b << 4), even[u]);
      e2m1_to_h2(select_bits(a >> 4, b), odd[u]);
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

// A unit's queries as the score MMAs take them: four registers for 32 elements of 8 rows, held in
// registers or (kQueriesInSmem) in the warp's shared memory, 16 bytes a lane.
template <int D, int NT, bool kSmem = Cfg<D, NT>::kQueriesInSmem>
struct Queries {
  uint32_t f[NT][D / 8];
  __device__ __forceinline__ void bind(uint32_t) {}
  __device__ __forceinline__ void put(int n, const uint32_t (&x)[D / 8]) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) f[n][i] = x[i];
  }
  __device__ __forceinline__ void get(int n, int w, uint32_t (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f[n][4 * w + i];
  }
};
template <int D, int NT>
struct Queries<D, NT, true> {
  uint32_t at; // the lane's
  __device__ __forceinline__ void bind(uint32_t a) { at = a; }
  __device__ __forceinline__ void put(int n, const uint32_t (&x)[D / 8]) {
#pragma unroll
    for (int i = 0; i < D / 8; i += 4)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (n * (D / 32) + i / 4) * 512), "r"(x[i]),
                   "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]));
  }
  __device__ __forceinline__ void get(int n, int w, uint32_t (&x)[4]) const { lds(at + (n * (D / 32) + w) * 512, x); }
};

// One tile from position pos. mapped: a bit for each 16 tokens, the first highest; masked: some row of the block does not see every token.
template <int D, int NT>
__device__ __forceinline__ void do_tile(uint32_t sm, const Reads<D> &at, const Queries<D, NT> &q,
                                        const float (&mul)[NT][2], const Kernel &k, int b, int row0, int pos,
                                        unsigned mapped, bool masked, int lane, Acc<D, NT> &acc) {
  constexpr int kScales = (D + 64) / 128;
  float s[kSub][NT][4];
  {
    Tile<D> t[kSub];
    uint32_t scale2[kSub][2][kScales]; // the scales of the lane's D/64 blocks, as fp16 pairs
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      read_keys<D>(sm + u * 18 * D, at, t[u]);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kScales; ++i) scale2[u][r][i] = e4m3_to_h2(t[u].ks[r] >> (16 * i));
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      uint32_t c[kSub][2][4];
      const uint32_t sel = w / 2 % 2 ? 0x3232u : 0x1010u; // the scale of this word's block, in both halves
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          e2m1_to_h2(t[u].k[r][w], c[u][r]);
          const uint32_t sc = prmt(scale2[u][r][w / 4], 0u, sel);
#pragma unroll
          for (int j = 0; j < 4; ++j) c[u][r][j] = hmul2(c[u][r][j], sc);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t f[4];
        q.get(n, w, f);
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          if (w == 0) mma16816_first(s[u][n], c[u][0][0], c[u][1][0], c[u][0][1], c[u][1][1], f[0], f[1]);
          else mma16816(s[u][n], c[u][0][0], c[u][1][0], c[u][0][1], c[u][1][1], f[0], f[1]);
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) mma16816(s[u][n], c[u][0][2], c[u][1][2], c[u][0][3], c[u][1][3], f[2], f[3]);
      }
    }
  }
  float x[kSub][NT][4]; // logits (log2 units) less the column's reference; -infinity: not seen
#pragma unroll
  for (int u = 0; u < kSub; ++u)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][n][e] = fmaf(s[u][n][e], mul[n][e & 1], -acc.ref[n][e & 1]);
  if (masked) {
    const int g = lane >> 2, tig = lane & 3;
    const Rows rows = rows_of(k, b);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int query = query_of(k, row0 + 8 * n + 2 * tig + c);
        const int limit = (query < rows.count ? rows.limit(query) : rows.seen) - pos - g;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          const bool here = mapped >> (kSub - 1 - u) & 1u;
          if (!here || 16 * u >= limit) x[u][n][c] = -INFINITY;
          if (!here || 16 * u + 8 >= limit) x[u][n][c + 2] = -INFINITY;
        }
      }
  }
  float top = -INFINITY;
#pragma unroll
  for (int u = 0; u < kSub; ++u)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, x[u][n][e]);
  if (__any_sync(0xffffffffu, top > kRefSlack)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int e = c; e < 4; e += 2) {
            s[u][n][e] = x[u][n][e] == -INFINITY ? x[u][n][e] : s[u][n][e] * mul[n][c];
            m = fmaxf(m, s[u][n][e]);
          }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = fmaxf(acc.ref[n][c], m - kRefDrop), f = softmax_exp2(acc.ref[n][c] - ref);
        acc.ref[n][c] = ref;
#pragma unroll
        for (int u = 0; u < kSub; ++u) x[u][n][c] = s[u][n][c] - ref, x[u][n][c + 2] = s[u][n][c + 2] - ref;
        acc.l[n][c] *= f;
        acc.l[n][c + 2] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc.o[n][i][c] *= f, acc.o[n][i][c + 2] *= f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kSub; ++u) {
    Tile<D> t;
    read_values<D>(sm + u * 18 * D, at, t);
    uint32_t p[NT][2]; // the weights as the value MMAs take them
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      p[n][0] = transpose8x8(pack_h2(softmax_exp2(x[u][n][0]), softmax_exp2(x[u][n][1])));
      p[n][1] = transpose8x8(pack_h2(softmax_exp2(x[u][n][2]), softmax_exp2(x[u][n][3])));
      mma16816(acc.l[n], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, p[n][0], p[n][1]);
    }
    if (masked) {
      // 0 * NaN is NaN: a token that a row does not see must not reach it through its scale either.
      // Tokens that no row sees get scale 0. A NaN scale among the rest of a masked tile is rare;
      // then each query of the block takes its own pass with only its own tokens and columns.
      const int g = lane >> 2, tig = lane & 3;
      const Rows rows = rows_of(k, b);
      const int token = pos + 16 * u + 2 * tig;
      const bool here = mapped >> (kSub - 1 - u) & 1u;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!here || token + (i >> 1) * 8 + (i & 1) >= rows.seen) t.vs[i] = 0u;
        nan |= (t.vs[i] & 0x7Fu) == 0x7Fu || (t.vs[i] & 0x7F00u) == 0x7F00u;
      }
      if (__any_sync(0xffffffffu, nan)) {
        const int last = min(query_of(k, row0 + 8 * NT - 1), rows.count - 1);
        for (int query = query_of(k, row0); query <= last; ++query) {
          const int lim = rows.limit(query);
          uint32_t pq[NT][2], vq[4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const bool mine = query_of(k, row0 + 8 * n + g) == query; // a fragment's column is row g
            pq[n][0] = mine ? p[n][0] : 0u;
            pq[n][1] = mine ? p[n][1] : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) vq[i] = token + (i >> 1) * 8 + (i & 1) < lim ? t.vs[i] : 0u;
          // columns of other queries still meet this pass's NaN scales, with weight 0
          unsigned own = 0;
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i)
            own |= static_cast<unsigned>(query_of(k, row0 + 8 * (i >> 1) + 2 * tig + (i & 1)) == query) << i;
          add_values<D, NT, true>(t, vq, pq, acc, own);
        }
        continue;
      }
    }
    add_values<D, NT, false>(t, t.vs, p, acc);
  }
}

constexpr int kCombineThreads = 256;

enum { kHead = 1, kHeadEnds = 2, kTail = 4, kSome = 8 }; // what a warp's stretch left behind

// Rows without a weight that see a mapped position of the stretch [begin, end) get kLost as their sum.
template <int D, int NT>
__device__ __forceinline__ void mark_lost(const Kernel &k, const Rows &rows, int b, int row0, int begin, int end,
                                          int lane, Acc<D, NT> &acc) {
  bool none = false;
#pragma unroll
  for (int n = 0; n < NT; ++n) none |= acc.l[n][0] == 0.0f || acc.l[n][1] == 0.0f;
  if (!__any_sync(0xffffffffu, none)) return;
  const int *entries = k.c.bt + static_cast<long long>(b) * k.c.maxp;
  const int pages = end > begin ? ((end - 1) >> k.c.pshift) + 1 : 0;
  int first = INT_MAX; // the first mapped position
#pragma unroll 1
  for (int j = begin >> k.c.pshift; j < pages; j += 32) {
    const int page = j + lane < pages ? __ldg(entries + j + lane) : -1;
    const unsigned hit = __ballot_sync(0xffffffffu, static_cast<unsigned>(page) < static_cast<unsigned>(k.c.num_pages));
    if (hit) {
      first = max((j + __ffs(hit) - 1) << k.c.pshift, begin);
      break;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (acc.l[n][c] == 0.0f && first < rows.limit(query_of(k, row0 + 8 * n + 2 * (lane & 3) + c))) acc.l[n][c] = kLost;
}

__device__ __forceinline__ float inverse_sum(const Kernel &k, float l) { // times the value scale; off by 2 units in the last place
  return l < kLostBelow ? __int_as_float(0x7FC00000) : __fdividef(k.c.g[1], l);
}

// Writes a warp's state as a partial.
template <int D, int NT>
__device__ __forceinline__ void store_partial(float *slot, const Acc<D, NT> &acc, int lane) {
  constexpr int R = 8 * NT;
  const int g = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * n + 2 * tig + c;
      if (g == 0) slot[R * D + 2 * r] = acc.ref[n][c], slot[R * D + 2 * r + 1] = acc.l[n][c];
#pragma unroll
      for (int i = 0; i < D / 16; i += 2)
        *reinterpret_cast<float4 *>(slot + r * D + g * (D / 8) + 2 * i) =
            make_float4(acc.o[n][i][c], acc.o[n][i][c + 2], acc.o[n][i + 1][c], acc.o[n][i + 1][c + 2]);
    }
}

__device__ __forceinline__ long long out_row(const Kernel &k, int b, int h, int row) {
  const int query = query_of(k, row);
  return (static_cast<long long>(b) * k.Lq + query) * k.Hq + h * k.G + row - query * k.G;
}

// Writes four elements of an output row from its sums. A sum of 0 means that every position was unmapped.
template <int D>
__device__ __forceinline__ void store_row(const Kernel &k, const Rows &rows, int b, int h, int row, int d, float l,
                                          const float4 &o) {
  const bool some = rows.limit(query_of(k, row)) > 0 && l != 0.0f;
  const float inv = inverse_sum(k, l);
  const long long at = out_row(k, b, h, row) * D + d;
  store_out(k, at, some ? o.x * inv : 0.0f, some ? o.y * inv : 0.0f);
  store_out(k, at + 2, some ? o.z * inv : 0.0f, some ? o.w * inv : 0.0f);
}

// Writes a unit that one warp has seen whole.
template <int D, int NT>
__device__ __forceinline__ void store_whole(const Kernel &k, const Rows &rows, int b, int h, int row0,
                                            const Acc<D, NT> &acc, int lane) {
  const int g = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = row0 + 8 * n + 2 * tig + c;
      if (row >= k.Lq * k.G) continue;
      const bool some = rows.limit(query_of(k, row)) > 0 && acc.l[n][c] != 0.0f; // as in store_row
      const float inv = some ? inverse_sum(k, acc.l[n][c]) : 0.0f;
      const size_t at = static_cast<size_t>(out_row(k, b, h, row) * D + g * (D / 8));
      float x[D / 8];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        x[2 * i] = some ? acc.o[n][i][c] * inv : 0.0f;
        x[2 * i + 1] = some ? acc.o[n][i][c + 2] * inv : 0.0f;
      }
      if (k.out_dtype == TQ_F32) {
        store_vec<D / 8>(k.out, TQ_F32, at, x);
      } else {
        uint32_t w[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          w[i] = k.out_dtype == TQ_BF16 ? *reinterpret_cast<const uint32_t *>(&v) : pack_h2(x[2 * i], x[2 * i + 1]);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(k.out) + at);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
    }
}

// Queries of a unit: row g of each column tile as fp16, and what turns the columns' scores into log2
// units. fp16 queries are taken as they are; bf16 rows are multiplied by the power of two that brings
// their largest element to 2^14..2^15 (2^126 at most: bf16 values are multiples of 2^-133).
template <int D, int NT>
__device__ __forceinline__ void load_queries(const Kernel &k, const Rows &rows, int b, int h, int row0, int lane,
                                             Queries<D, NT> &queries, float (&mul)[NT][2]) {
  const int g = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = row0 + 8 * n + g;
    uint32_t q[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) q[i] = 0u;
    if (query_of(k, row) < rows.count) {
      const uint4 *src = reinterpret_cast<const uint4 *>(k.q + out_row(k, b, h, row) * D + tig * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = __ldg(src + i);
        q[4 * i] = v.x, q[4 * i + 1] = v.y, q[4 * i + 2] = v.z, q[4 * i + 3] = v.w;
      }
    }
    int e = 0;
    if (k.bf16) {
      uint32_t top = 0; // the largest magnitude in each half, as bits; infinities and NaN stand above
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, q[i] & 0x7FFF7FFFu);
      top = max(top >> 16, top & 0xFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int field = top >> 7; // of the exponent
      e = top == 0 || field == 255 ? 0 : min(141 - field, 126);
      const float f = __uint_as_float((127 + e) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) q[i] = pack_h2(bf16_lo(q[i]) * f, bf16_hi(q[i]) * f);
    }
    queries.put(n, q);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int ec = __shfl_sync(0xffffffffu, e, (2 * tig + c) * 4);
      mul[n][c] = k.scale * __uint_as_float((127 - ec) << 23) * k.klog;
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas) mx_decode_kernel(const Kernel k) {
  using C = Cfg<D, NT>;
  constexpr int R = 8 * NT, W = kWarps, S = C::kStages;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint32_t s_scan[W], s_bound[W + 1], s_ahead[W];
  __shared__ int s_b0[W], s_left[W];
  __shared__ int4 s_tail[W];
  __shared__ Rows s_rows[W]; // of the tails
  __shared__ Cursor s_copy[W], s_done[W]; // where the warps' copies and sums are (out of the registers' way)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // ---- the warps' stretches of the weighted tile space
  const int B = k.c.B, per = (B + kThreads - 1) / kThreads;
  const int units = k.c.Hkv * k.row_blocks; // of a sequence
  uint32_t mine = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < B) {
      const int nt = tiles_of(k, tid * per + i);
      mine += nt ? (nt + kUnitCost) * units : 0;
    }
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int cta = blockIdx.x;
  const Split split(total, gridDim.x, W);
  if (tid <= W) s_bound[tid] = split.begin(cta * W + tid);
  if (tid < W) s_b0[tid] = 0, s_ahead[tid] = 0;
  __syncthreads();
  uint32_t at = before + incl - mine;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= B) break;
    const int nt = tiles_of(k, b);
    if (nt == 0) continue;
    const uint32_t len = (nt + kUnitCost) * units;
    if (at <= s_bound[W - 1] && at + (len - 1) >= s_bound[0])
      for (int w = 0; w < W; ++w)
        if (s_bound[w] >= at && s_bound[w] - at < len) s_b0[w] = b, s_ahead[w] = s_bound[w] - at;
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
  const int len = static_cast<int>(s_bound[warp + 1] - s_bound[warp]);
  uint8_t *ring = sm + warp * C::kWarpBytes;
  int left = 0;
  if (len > 0) {
    const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // ---- copies run S - 1 tiles ahead
    // the lane's 16 bytes of the next tile: `chunk` in the codes, `schunk` in the scales (keys' in the first
    // half of D/8 lanes, values' in the second; further lanes repeat them)
    const uint8_t *sc = k.c.scales[lane / (D / 16) & 1];
    const uint32_t swz = __shfl_sync(0xffffffffu, (lane >> 3) * 128 + (((lane & 7) ^ chunk_swizzle<D>(lane >> 3)) << 4), lane);
    const uint32_t sdst = __shfl_sync(0xffffffffu, 16 * D + (lane & (D / 8 - 1)) * 16, lane);
    uint32_t chunk = 0, schunk = 0;
    const int page_tiles = 1 << (k.c.pshift - 4);
    const int *entry = nullptr;  // table entry behind next_page's
    int run = 0, left_tiles = 0; // 16-token tiles left on the current page, and of the unit's behind it
    int next_page = -1;          // the page behind the current one, read ahead
    uint32_t head;               // first record of the head in page 0
    unsigned mapped = 0, ok = 0; // a bit for each 16 tokens copied, the latest lowest; all or none for the current page
    // Unmapped pages, and what is behind the stretch's end, copy records of page 0: never looked at, and
    // cheaper than a branch for every tile.
    auto enter_page = [&](int in_page) {
      ok = static_cast<unsigned>(next_page) < static_cast<unsigned>(k.c.num_pages) ? (1u << kSub) - 1u : 0u;
      // 16-byte chunks of codes < 2^32 (the host checks), so their index is one 32-bit word
      const uint32_t rec = ok ? ((next_page * static_cast<uint32_t>(k.c.Hkv)) << k.c.pshift) + head + (in_page << 4) : 0u;
      chunk = rec * (D / 32) + lane;
      schunk = (rec >> 4) * (D / 16) + (lane & (D / 16 - 1));
      run = page_tiles - in_page;
      if (left_tiles > 0) {
        run = min(run, left_tiles);
        left_tiles -= run;
        if (left_tiles > 0) next_page = __ldg(entry++);
      }
    };
    {
      Cursor c;
      c.start(k, s_b0[warp], s_ahead[warp]);
      s_done[warp] = s_copy[warp] = c;
      const int tile = kSub * c.first();
      left_tiles = max(c.end16(k, len) - tile, 0); // 0: the stretch begins with the cost of a unit
      entry = k.c.bt + static_cast<long long>(c.b) * k.c.maxp + (tile >> (k.c.pshift - 4));
      head = static_cast<uint32_t>(c.h) << k.c.pshift;
      if (left_tiles > 0) {
        next_page = __ldg(entry++);
        enter_page(tile & (page_tiles - 1));
      }
    }
    __syncwarp();
    auto copy = [&](uint32_t dst, auto subs) { // subs x 16 adjacent tokens
      const uint8_t *a = k.c.codes[0] + static_cast<size_t>(chunk) * 16, *b = k.c.codes[1] + static_cast<size_t>(chunk) * 16;
      const uint8_t *s = sc + static_cast<size_t>(schunk) * 16;
#pragma unroll
      for (int u = 0; u < subs.value; ++u) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) { // 512 bytes: the swizzle of lines 4 apart differs for D = 256 only
          const uint32_t to = dst + u * C::kSixteen + (D == 256 ? swz ^ ((j & 1) << 6) : swz) + j * 512;
          copy16(to, a + u * 8 * D + j * 512);
          copy16(to + 8 * D, b + u * 8 * D + j * 512);
        }
        copy16(dst + u * C::kSixteen + sdst, s + u * D);
      }
      chunk += subs.value * (D / 2);
      schunk += subs.value * (D / 16);
    };
    auto copy16_tokens = [&](uint32_t dst) {
      if (run == 0) {
        if (left_tiles == 0) { // the next unit with tiles in the stretch
          Cursor c = s_copy[warp];
          bool more;
          do more = c.next(k, len);
          while (more && c.end(len) == 0);
          next_page = -1;
          if (more) {
            left_tiles = c.end16(k, len);
            entry = k.c.bt + static_cast<long long>(c.b) * k.c.maxp;
            head = static_cast<uint32_t>(c.h) << k.c.pshift;
            next_page = __ldg(entry++);
          }
          __syncwarp();
          s_copy[warp] = c;
          __syncwarp();
        }
        enter_page(0);
      }
      copy(dst, std::integral_constant<int, 1>{});
      --run;
      mapped = 2 * mapped + (ok & 1u);
    };
    auto copy_tile = [&](uint32_t dst) {
      if (run >= kSub) { // within a page
        copy(dst, std::integral_constant<int, kSub>{});
        run -= kSub;
        mapped = (mapped << kSub) | ok;
      } else {
        copy16_tokens(dst);
#pragma unroll 1
        for (int u = 1; u < kSub; ++u) {
          if (run | left_tiles) copy16_tokens(dst + u * C::kSixteen);
          else mapped *= 2; // the unit has ended
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy_tile(ring_addr + i * C::kTile);
    const Reads<D> reads(lane);
    int at_stage = 0, free_stage = (S - 1) * C::kTile; // byte offsets of the next tile and of the next copy
    left = kSome;
    bool more;
    do {
      const Cursor cu = s_done[warp];
      const int t0 = cu.first(), t1 = cu.end(len);
      if (t0 < t1) { // else only the cost of a unit lies in the stretch
        const int b = cu.b, h = cu.h, row0 = cu.rb * R;
        Queries<D, NT> q; // each lane reads what it wrote
        q.bind(ring_addr + S * C::kTile + lane * 16);
        float mul[NT][2];
        int full; // every row of the block sees the positions below
        {
          const Rows rows = rows_of(k, b);
          load_queries<D, NT>(k, rows, b, h, row0, lane, q, mul);
          const int query = query_of(k, row0);
          full = query < rows.count ? rows.limit(query) : rows.seen;
        }
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
        for (int tile = t0; tile < t1; ++tile) {
          asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
          __syncwarp(); // all lanes' copies of this tile are there, and the oldest stage's readers are done
          copy_tile(ring_addr + free_stage);
          constexpr int kTokens = 16 * kSub;
          constexpr unsigned kAll = (1u << kSub) - 1u;
          const unsigned here = mapped >> (kSub * (S - 1)) & kAll;
          const int pos = tile * kTokens;
          do_tile<D, NT>(ring_addr + at_stage, reads, q, mul, k, b, row0, pos, here, pos + kTokens > full || here != kAll, lane, acc);
          free_stage = at_stage;
          at_stage = at_stage + C::kTile == S * C::kTile ? 0 : at_stage + C::kTile;
        }
        {
          constexpr int kTokens = 16 * kSub;
          const Rows rows = rows_of(k, b);
          mark_lost<D, NT>(k, rows, b, row0, t0 * kTokens, min(t1 * kTokens, rows.seen), lane, acc);
        }
        if (t0 > 0) {
          left |= kHead | (t1 == cu.nt ? kHeadEnds : 0);
          store_partial<D, NT>(reinterpret_cast<float *>(ring + C::kHeadAt), acc, lane);
        } else if (t1 == cu.nt) {
          store_whole<D, NT>(k, rows_of(k, b), b, h, row0, acc, lane);
        } else { // the last unit of the stretch: its partial takes the ring's place
          left |= kTail;
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          __syncwarp();
          store_partial<D, NT>(reinterpret_cast<float *>(ring), acc, lane);
          if (lane == 0) {
            const uint32_t last = s_bound[warp] + cu.at + cu.nt - 1; // the unit's last tile, in the whole space
            const int parts = static_cast<int>(min(split.share_of(last) / W, gridDim.x - 1u)) - cta + 1;
            s_tail[warp] = make_int4(b, h, row0, max(parts, 1));
            s_rows[warp] = rows_of(k, b);
          }
        }
      }
      Cursor c = s_done[warp];
      more = c.next(k, len);
      __syncwarp();
      s_done[warp] = c;
      __syncwarp();
    } while (more);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  pdl_trigger();
  if (lane == 0) s_left[warp] = left;
  __syncthreads();
  // ---- join the warps' partials: a cut unit is the tail of one warp and the heads of those behind it
  unsigned some = 0, heads = 0, ends = 0, tails = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int l = s_left[w];
    some |= (l & kSome ? 1u : 0u) << w, heads |= (l & kHead ? 1u : 0u) << w;
    ends |= (l & kHeadEnds ? 1u : 0u) << w, tails |= (l & kTail ? 1u : 0u) << w;
  }
  constexpr int kPer = 4; // adjacent elements of a row that a thread joins at a time
  bool goes_on = false;
#pragma unroll 1
  for (int first = -1; first < W; ++first) { // -1: the unit that CTAs before this one began
    if (first >= 0 && !(tails >> first & 1u)) continue;
    // the heads behind: up to the first that ends the unit, or before the first warp that begins with another
    const unsigned behind = ~0u << (first + 1);
    const unsigned stop = behind & (ends | (some & ~heads));
    unsigned parts = heads & behind & (stop ? (stop & ~(stop - 1)) * 2 - 1 : ~0u);
    if (first < 0 && parts == 0) continue;
    const bool whole = first >= 0 && (parts & ends);
    goes_on |= first >= 0 && !whole;
    if (first >= 0) parts |= 1u << first;
    if (first >= 0 && !whole && tid == 0) k.desc[cta] = s_tail[first];
    float *dst = k.part + (2ll * cta + (first >= 0)) * (C::kSlot / 4);
#pragma unroll 1
    for (int i = tid * kPer; i < R * D; i += kThreads * kPer) {
      const int r = i / D;
      const float *src[W];
      float2 st[W]; // references and sums
      float ref = kRefEmpty;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        src[w] = reinterpret_cast<const float *>(sm + w * C::kWarpBytes + (w == first ? 0 : C::kHeadAt));
        st[w] = parts >> w & 1u ? *reinterpret_cast<const float2 *>(src[w] + R * D + 2 * r) : make_float2(kRefEmpty, 0.0f);
        ref = fmaxf(ref, st[w].x);
      }
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (parts >> w & 1u) {
          const float f = softmax_exp2(st[w].x - ref);
          const float4 v = *reinterpret_cast<const float4 *>(src[w] + i);
          l = fmaf(f, st[w].y, l);
          o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
        }
      if (whole) {
        const int row = s_tail[first].z + r;
        if (row >= k.Lq * k.G) continue;
        store_row<D>(k, s_rows[first], s_tail[first].x, s_tail[first].y, row, i % D, l, o);
      } else {
        *reinterpret_cast<float4 *>(dst + i) = o;
        if (i % D == 0) *reinterpret_cast<float2 *>(dst + R * D + 2 * r) = make_float2(ref, l);
      }
    }
  }
  if (tid == 0 && !goes_on) k.desc[cta] = make_int4(0, 0, 0, 0);
}

// Joins the partials of a unit that several CTAs share: parts 0 (slot 1 of its first CTA) and
// 1.. (slot 0 of the CTAs behind it). One CTA for each boundary; most return at once.
template <int D, int NT>
__global__ void __launch_bounds__(kCombineThreads) mx_combine_kernel(const Kernel k) {
  constexpr int R = 8 * NT, kSlot = Cfg<D, NT>::kSlot / 4;
  pdl_wait();
  const int cta = blockIdx.x;
  const int4 d = k.desc[cta];
  if (d.w == 0) return;
  const int parts = d.w;
  const Rows rows = rows_of(k, d.x);
  const float *first = k.part + (2ll * cta + 1) * kSlot, *rest = k.part + 2ll * cta * kSlot; // part p > 0: rest + 2 p slots
#pragma unroll 1
  for (int i = threadIdx.x * 4; i < R * D; i += kCombineThreads * 4) {
    const int r = i / D;
    if (d.z + r >= k.Lq * k.G) break;
    float2 st = *reinterpret_cast<const float2 *>(first + R * D + 2 * r);
    float4 o = *reinterpret_cast<const float4 *>(first + i);
    float ref = st.x, l = st.y;
#pragma unroll 4
    for (int p = 1; p < parts; ++p) { // the first part's sums are scaled along
      const float *s = rest + 2ll * p * kSlot;
      st = *reinterpret_cast<const float2 *>(s + R * D + 2 * r);
      const float4 v = *reinterpret_cast<const float4 *>(s + i);
      const float now = fmaxf(ref, st.x), back = softmax_exp2(ref - now), f = softmax_exp2(st.x - now);
      ref = now;
      l = fmaf(f, st.y, l * back);
      o.x = fmaf(f, v.x, o.x * back), o.y = fmaf(f, v.y, o.y * back);
      o.z = fmaf(f, v.z, o.z * back), o.w = fmaf(f, v.w, o.w * back);
    }
    store_row<D>(k, rows, d.x, d.y, d.z + r, i % D, l, o);
  }
}

template <int D, int NT>
cudaError_t run(const Kernel &k, const MxPlan &p, cudaStream_t s) {
  constexpr int smem = Cfg<D, NT>::kSmem;
  static std::atomic<uint64_t> set{0}; // devices (the first 64) whose kernel has its shared memory size
  const uint64_t bit = p.device < 64 ? 1ull << p.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(mx_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_release);
  }
  e = launch_pdl(mx_decode_kernel<D, NT>, dim3(p.ctas), dim3(kThreads), smem, s, k);
  if (e != cudaSuccess) return e;
  return launch_pdl(mx_combine_kernel<D, NT>, dim3(p.ctas), dim3(kCombineThreads), 0, s, k);
}

template <class F>
auto with_shape(int d, int nt, F &&f) { // f.operator()<D, NT>()
  if (d == 64) return nt == 1 ? f.template operator()<64, 1>() : f.template operator()<64, 2>();
  if (d == 128) return nt == 1 ? f.template operator()<128, 1>() : f.template operator()<128, 2>();
  return f.template operator()<256, 1>();
}

struct Ctas { // of an SM
  template <int D, int NT>
  int operator()() const { return Cfg<D, NT>::kCtas; }
};
struct Launch {
  const Kernel &k;
  const MxPlan &p;
  cudaStream_t s;
  template <int D, int NT>
  cudaError_t operator()() const { return run<D, NT>(k, p, s); }
};

} // namespace

MxPlan plan_mx_decode(int Hkv, int d, int Hq, int Lq, int device, int sm_count) {
  MxPlan p;
  p.device = device;
  // A block of 16 rows takes about 1.6 times as long as one of 8 (operands are made once for both), so it
  // is taken where it halves the blocks or nearly so: 16 rows of 8 x 9001 positions 37.8 us against 42.9,
  // 128 rows of 8 x 4000 93 against 118, but 20 rows, 700..9001 positions, 32.1 against 29.3 in three
  // blocks of 8. (24 rows a block: 33.9 us there, 94.8 us for 128 rows.) Heads of 256 leave room for one.
  const int rows = Lq * (Hq / Hkv), of8 = (rows + 7) / 8, of16 = (rows + 15) / 16, most = d == 256 ? 1 : 2;
  p.nt = most == 2 && 5 * of8 >= 8 * of16 ? 2 : 1;
  p.row_blocks = p.nt == 2 ? of16 : of8;
  p.ctas = sm_count * with_shape(d, p.nt, Ctas{});
  // one size serves every number of queries and heads: the larger of the block sizes'
  p.ws_bytes = 0;
  for (int nt = 1; nt <= most; ++nt) {
    const size_t ctas = static_cast<size_t>(sm_count) * with_shape(d, nt, Ctas{});
    p.ws_bytes = std::max(p.ws_bytes, ctas * (2 * 8 * nt * (d + 2) * sizeof(float) + sizeof(int4)));
  }
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
  k.inv_group = 1.0f / static_cast<float>(k.G);
  k.Lq = a.Lq;
  k.row_blocks = a.plan.row_blocks;
  k.bf16 = a.dtype == TQ_BF16;
  k.out_dtype = a.out_dtype;
  k.scale = a.scale;
  k.klog = 1.4426950408889634f * a.c.g[0];
  return with_shape(a.c.d, a.plan.nt, Launch{k, a.plan, s});
}

} // namespace tq
