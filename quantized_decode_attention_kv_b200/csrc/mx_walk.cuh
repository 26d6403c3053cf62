// How the warps of the microscaled attention divide and walk the weighted tile space: integer arithmetic
// on lengths, counts and shapes, which compiles for the device and, for its tests, on the host. K is any
// struct with the cache (c.B, c.Hkv, c.maxp, c.pshift), lens, counts, Lq and row_blocks.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MX_FN __device__ __forceinline__
#else
#include <algorithm>
#define MX_FN inline
#endif

namespace tq {
namespace mx {

#ifndef __CUDACC__
using std::max;
using std::min;
inline int __ldg(const int *p) { return *p; }
#endif

MX_FN int clamp_count(const int *counts, int b, int rows) {
  return counts ? min(max(__ldg(counts + b), 0), rows) : rows;
}

// What a unit costs besides its tiles, in tiles. 1, 2, 4: ragged batch of 32 27.3, 24.9, 24.3 us; 512 units
// of 20 positions 9.0, 10.3, 12.0 us.
constexpr int kUnitCost = 2;
constexpr int kMinTiles = 2; // tiles a warp gets at least, unit costs included (2, 4: 333 positions 9.8, 12.2 us)
constexpr int kSub = 2;      // 16-token MMA tiles of a tile

template <class K>
MX_FN int tiles_of(const K &k, int b) {
  if (clamp_count(k.counts, b, k.Lq) == 0) return 0;
  const int cap = k.c.maxp << k.c.pshift;
  return (min(max(__ldg(k.lens + b), 0), cap) + 16 * kSub - 1) / (16 * kSub);
}
// Position limits of a row of a unit: row r is query r / G, head r % G of the group; it sees
// positions below limit(r) (0: none).
struct Rows {
  int count, first, seen; // queries of the sequence, position of query 0, cached positions
  MX_FN int limit(int query) const {
    return query < count ? min(max(first + query + 1, 0), seen) : 0;
  }
};
template <class K>
MX_FN Rows rows_of(const K &k, int b) {
  Rows r;
  const int len = __ldg(k.lens + b), cap = k.c.maxp << k.c.pshift;
  r.count = clamp_count(k.counts, b, k.Lq);
  r.first = len - r.count;
  r.seen = min(max(len, 0), cap);
  return r;
}

// A warp's way through its stretch of the weighted tile space: units one after the other. Positions
// are relative to the stretch's begin. (Lengths that another stream changes while the kernel runs make
// wrong outputs, never indexes out of range: sequences and heads are bounded here, CTAs at the joins.)
struct Cursor {
  int b, nt, h, rb; // sequence, its tiles, KV head, row block
  int at;           // position of the unit's first tile
  template <class K>
  MX_FN void start(const K &k, int b0, uint32_t ahead) { // ahead: begin less b0's begin
    b = b0;
    nt = tiles_of(k, b);
    const uint32_t unit = min(ahead / (nt + kUnitCost), static_cast<uint32_t>(k.c.Hkv * k.row_blocks - 1));
    at = static_cast<int>(unit * (nt + kUnitCost) - ahead) + kUnitCost;
    h = unit / k.row_blocks;
    rb = unit - h * k.row_blocks;
  }
  MX_FN int first() const { return max(-at, 0); }
  MX_FN int end(int len) const { return min(max(len - at, 0), nt); }
  // 16-token tiles from the unit's begin to its end within the stretch
  template <class K>
  MX_FN int end16(const K &k, int len) const {
    return min(kSub * end(len), (rows_of(k, b).seen + 15) >> 4);
  }
  // the next unit that begins within the stretch; false at its end, and from then on: the copies run ahead
  // of the sums and ask again. (Lengths that shrank meanwhile end the sequences before the stretch.)
  template <class K>
  MX_FN bool next(const K &k, int len) {
    at += nt + kUnitCost;
    if (at - kUnitCost >= len || b >= k.c.B) return false;
    if (++rb < k.row_blocks) return true;
    rb = 0;
    if (++h < k.c.Hkv) return true;
    h = 0;
    do {
      if (++b >= k.c.B) return false;
      nt = tiles_of(k, b);
    } while (nt == 0);
    return true;
  }
};

// The weighted tile space (below 2^32: the host checks) over the warps of the CTAs that take part:
// the first `more` shares are one longer than the others.
struct Split {
  uint32_t total, each, more;
  MX_FN Split(uint32_t n, int ctas, int warps) {
    total = n;
    const uint32_t shares = min(static_cast<uint32_t>(ctas), max(n / (warps * kMinTiles), 1u)) * warps;
    each = n / shares;
    more = n - each * shares;
  }
  MX_FN uint32_t begin(uint32_t i) const { // shares behind the last one begin at the end
    const uint64_t at = static_cast<uint64_t>(i) * each + min(i, more);
    return at < total ? static_cast<uint32_t>(at) : total;
  }
  MX_FN uint32_t share_of(uint32_t at) const {
    const uint32_t bend = more * (each + 1);
    return at < bend ? at / (each + 1) : more + (at - bend) / each;
  }
};

} // namespace mx
} // namespace tq
