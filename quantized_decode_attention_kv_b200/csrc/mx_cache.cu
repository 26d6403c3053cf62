// Write and read of the microscaled 4-bit paged cache.
//
// Write: a block of 16 elements x has the scale byte S = E4M3(min(max|x| / (6 g), 448)) and the
// codes E2M1(x / (S g)), both to nearest with ties to even; a NaN or infinity in the block makes
// S NaN (0x7F, codes 0), so that it stays visible. Read: E2M1 * S * g, one rounding in fp32 and
// one to the output's type.
//
// Both stream: a thread owns one block of U rows of a head (two 16-byte loads of 16-bit input, 9 bytes
// out), so a row's blocks and the rows of one head are contiguous across a warp, and nothing is kept
// between threads. HBM bounds them (write: 2 + 9/16 bytes an element) only while a block takes about
// 150 instructions, so those are counted: grids without divisions, record numbers of 32 bits, the
// maximum on packed 16-bit patterns, packed fp32 pairs (16 x 8 x 4096 rows of bf16, 344 MB each way,
// 53 us at the copy rate: write 98 -> 62 us, read 80 -> 60 us). A read back into padded rows mostly
// writes zeros, and plain writes reach half the copy rate: 134 MB take 37 us in a fill, and 35 us
// here with the write of 10 MB before them.
//
// Ties are common (16-bit inputs over a 4-bit scale hit an E2M1 midpoint m about once in 64), so
// x / (S g) has to land on the right side of them; x times r = 1 / (S g) alone does not.
//  - In general each quotient is corrected by its exact remainder: q = x r, q + (x - q S g) r is the
//    correctly rounded quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
//    System/6000", 1990).
//  - 16-bit inputs and a power of two g: x has at most 11 significant bits and m S g at most 7, so
//    |x / (S g) - m| is 0 or at least 2^-11 m >= 2^-13. x r is off by at most 8 * 2^-24; one FMA
//    x r + 768 rounds it to a multiple of 2^-14, which makes ties exact and leaves all else on its
//    side.
#include <cmath>

#include "mx.cuh"

namespace tq {
namespace {

using namespace mx;

constexpr int kThreads = 256;

// Which (sequence, head, block) and first row a thread owns. Bulk calls: a CTA takes U times kRows
// consecutive rows of one head, the grid is (rows, heads of keys and values, sequences). Small calls
// (one new token): 2^tshift rows of each of some heads, the grid is (heads of all sequences, 1, keys
// and values).
struct RowIndex {
  int which, b, h, t, blk;
  bool ok;
};

template <int D, bool kBulk, int U>
__device__ __forceinline__ RowIndex row_index(const MxRowsArgs &a, int tshift) {
  constexpr int kPer = D / kBlock, kRows = kThreads / kPer;
  const int r = threadIdx.x / kPer;
  RowIndex i;
  i.blk = threadIdx.x % kPer;
  if constexpr (kBulk) {
    const int head = blockIdx.y;
    const bool second = head >= a.c.Hkv;
    i.which = second || !a.x[0];
    i.h = head - (second ? a.c.Hkv : 0);
    i.b = blockIdx.z;
    i.t = blockIdx.x * (U * kRows) + r;
    i.ok = i.t < a.T;
  } else {
    const int bh = static_cast<int>(blockIdx.x) * (kRows >> tshift) + (r >> tshift);
    i.which = blockIdx.z || !a.x[0];
    i.t = r & ((1 << tshift) - 1);
    i.b = bh / a.c.Hkv;
    i.h = bh - i.b * a.c.Hkv;
    i.ok = i.b < a.c.B && i.t < a.T;
  }
  return i;
}

__device__ __forceinline__ uint32_t dup_low(uint32_t h) { return __byte_perm(h, 0u, 0x1010u); } // the low half twice

// Records of the thread's rows: kNone where a row is none of the sequence's, or not on a mapped page.
// (Codes are at most 64 GiB, so records are below 2^31.) Returns the number of rows of the sequence.
constexpr uint32_t kNone = 0xFFFFFFFFu;
template <int D, int U>
__device__ __forceinline__ int find_rows(const MxRowsArgs &a, const RowIndex &i, uint32_t (&rec)[U]) {
  constexpr int kRows = kThreads / (D / kBlock);
  const int n = clamp_count(a.counts, i.b, a.T);
  const long long first = static_cast<long long>(__ldg(a.lens + i.b)) - n + i.t;
  const int *row = a.c.bt + static_cast<long long>(i.b) * a.c.maxp;
  const uint32_t cap = static_cast<uint32_t>(a.c.maxp) << a.c.pshift; // <= 2^30
  int page[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long p = first + u * kRows;
    const bool here = i.t + u * kRows < n && p >= 0 && p < cap;
    rec[u] = here ? static_cast<uint32_t>(p) : 0u;
    page[u] = here ? __ldg(row + (rec[u] >> a.c.pshift)) : -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    rec[u] = static_cast<uint32_t>(page[u]) < static_cast<uint32_t>(a.c.num_pages)
                 ? ((static_cast<uint32_t>(page[u]) * a.c.Hkv + i.h) << a.c.pshift) + (rec[u] & ((1u << a.c.pshift) - 1u))
                 : kNone;
  return n;
}

// kPow2: 16-bit inputs and tensor scales that are powers of two.
template <int D, int DT, bool kBulk, int U, bool kPow2>
__global__ void __launch_bounds__(kThreads) mx_write_kernel(const MxRowsArgs a, int tshift) {
  constexpr int kRows = kThreads / (D / kBlock), kSize = DT == TQ_F32 ? 4 : 2, kVecs = kBlock * kSize / 16;
  pdl_wait();
  const RowIndex i = row_index<D, kBulk, U>(a, tshift);
  if (!i.ok) return;
  uint32_t rec[U];
  const int n = find_rows<D, U>(a, i, rec);
  if (i.t >= n) return;
  const long long *st = a.st[i.which];
  const char *src = static_cast<const char *>(a.x[i.which]) +
                    (i.b * st[0] + i.h * st[1] + i.t * st[2] + i.blk * kBlock) * kSize;
  uint4 raw[U][kVecs];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      raw[u][k] = i.t + u * kRows < n ? __ldg(reinterpret_cast<const uint4 *>(src + u * kRows * st[2] * kSize) + k)
                                      : make_uint4(0u, 0u, 0u, 0u);
  const float g = a.c.g[i.which], six = 6.0f * g, inv = a.inv6g[i.which];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (rec[u] == kNone) continue;
    uint32_t w[4 * kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      w[4 * k] = raw[u][k].x, w[4 * k + 1] = raw[u][k].y, w[4 * k + 2] = raw[u][k].z, w[4 * k + 3] = raw[u][k].w;
    // the largest |x| as bits: NaN and infinity compare above every finite value
    uint32_t bits = 0;
    float top;
    bool finite;
    if constexpr (DT == TQ_F32) {
#pragma unroll
      for (int k = 0; k < kBlock; ++k) bits = max(bits, w[k] & 0x7FFFFFFFu);
      top = __uint_as_float(bits);
      finite = bits < 0x7F800000u;
    } else {
#pragma unroll
      for (int k = 0; k < kBlock / 2; ++k) bits = __vmaxu2(bits, w[k] & 0x7FFF7FFFu);
      bits = max(bits >> 16, bits & 0xFFFFu);
      top = DT == TQ_BF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
      finite = bits < (DT == TQ_BF16 ? 0x7F80u : 0x7C00u);
    }
    uint32_t s = 0x7Fu;
    uint2 codes = make_uint2(0u, 0u);
    if (finite) {
      const float t0 = top * inv, t = fmaf(fmaf(-t0, six, top), inv, t0); // top / (6 g)
      s = float_to_e4m3(fminf(t, 448.0f));
      const float step = e4m3_to_float(s) * g;
      if (s != 0) {
        const float r = __frcp_rn(step);
        f2_t v[kBlock / 2];
#pragma unroll
        for (int k = 0; k < kBlock / 2; ++k) {
          if constexpr (DT == TQ_F32) {
            v[k] = f2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
          } else if constexpr (DT == TQ_BF16) {
            v[k] = f2(bf16_lo(w[k]), bf16_hi(w[k]));
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            v[k] = f2(f.x, f.y);
          }
        }
        if (!(t <= 448.0f)) { // saturated (NaN: top / (6 g) passes fp32): larger elements are 6 all the same
#pragma unroll
          for (int k = 0; k < kBlock / 2; ++k) {
            float x, y;
            f2_split(v[k], x, y);
            v[k] = f2(fminf(fmaxf(x, -7.0f * step), 7.0f * step), fminf(fmaxf(y, -7.0f * step), 7.0f * step));
          }
        }
        const f2_t r2 = f2(r, r), step2 = f2(-step, -step), magic = f2(768.0f, 768.0f), back = f2(-768.0f, -768.0f);
        float q[kBlock];
#pragma unroll
        for (int k = 0; k < kBlock / 2; ++k) {
          if constexpr (kPow2) {
            v[k] = add2(fma2(v[k], r2, magic), back);
          } else {
            const f2_t u2 = mul2(v[k], r2);
            v[k] = fma2(fma2(u2, step2, v[k]), r2, u2);
          }
          f2_split(v[k], q[2 * k], q[2 * k + 1]);
        }
        codes.x = float_to_e2m1(q);
        codes.y = float_to_e2m1(q + 8);
      }
    }
    *reinterpret_cast<uint2 *>(a.c.codes[i.which] + static_cast<size_t>(rec[u]) * (D / 2) + i.blk * 8) = codes;
    a.c.scales[i.which][static_cast<size_t>(rec[u]) * (D / kBlock) + i.blk] = static_cast<uint8_t>(s);
  }
}

template <int D, int DT, bool kBulk, int U>
__global__ void __launch_bounds__(kThreads) mx_read_kernel(const MxRowsArgs a, int tshift) {
  constexpr int kRows = kThreads / (D / kBlock), kSize = DT == TQ_F32 ? 4 : 2;
  pdl_wait();
  const RowIndex i = row_index<D, kBulk, U>(a, tshift);
  if (!i.ok) return;
  uint32_t rec[U];
  find_rows<D, U>(a, i, rec);
  uint2 codes[U];
  uint32_t s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    codes[u] = make_uint2(0u, 0u);
    s[u] = 0;
    if (rec[u] == kNone) continue;
    codes[u] = __ldg(reinterpret_cast<const uint2 *>(a.c.codes[i.which] + static_cast<size_t>(rec[u]) * (D / 2) + i.blk * 8));
    s[u] = __ldg(a.c.scales[i.which] + static_cast<size_t>(rec[u]) * (D / kBlock) + i.blk);
  }
  const long long *st = a.st[i.which];
  char *dst = static_cast<char *>(a.x[i.which]) + (i.b * st[0] + i.h * st[1] + i.t * st[2] + i.blk * kBlock) * kSize;
  const f2_t g = f2(a.c.g[i.which], a.c.g[i.which]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (i.t + u * kRows >= a.T) break;
    uint32_t out[kBlock * kSize / 4];
#pragma unroll
    for (int k = 0; k < kBlock * kSize / 4; ++k) out[k] = 0u;
    if (rec[u] != kNone) {
      const uint32_t scale = dup_low(e4m3_to_h2(s[u])), w[2] = {codes[u].x, codes[u].y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[4];
        e2m1_to_h2(w[k], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) { // E2M1 * S is exact in fp16
          const __half2 e = __hmul2(*reinterpret_cast<const __half2 *>(&h[j]), *reinterpret_cast<const __half2 *>(&scale));
          const float2 f = __half22float2(e);
          float x, y;
          f2_split(mul2(f2(f.x, f.y), g), x, y);
          if constexpr (DT == TQ_F32) {
            out[8 * k + 2 * j] = __float_as_uint(x);
            out[8 * k + 2 * j + 1] = __float_as_uint(y);
          } else if constexpr (DT == TQ_BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            out[4 * k + j] = *reinterpret_cast<const uint32_t *>(&p);
          } else {
            const __half2 p = __floats2half2_rn(x, y);
            out[4 * k + j] = *reinterpret_cast<const uint32_t *>(&p);
          }
        }
      }
    }
    // Lanes 2m and 2m + 1 hold neighbouring blocks: they swap halves of their 32-byte sectors, so that
    // each store of the warp writes whole sectors (first the even lane's, then the odd lane's).
    const unsigned pair = 3u << (threadIdx.x & 30);
    const bool odd = threadIdx.x & 1;
    char *to = dst + u * kRows * st[2] * kSize + (odd ? 16 - kBlock * kSize : 0); // the even lane's block
#pragma unroll
    for (int k = 0; k < kBlock * kSize / 4; k += 8) {
      uint32_t even_half[4], odd_half[4]; // what this lane writes of the even and of the odd lane's sector
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(pair, odd ? out[k + e] : out[k + 4 + e], 1);
        even_half[e] = odd ? got : out[k + e];
        odd_half[e] = odd ? out[k + 4 + e] : got;
      }
      const uint4 x = make_uint4(even_half[0], even_half[1], even_half[2], even_half[3]);
      const uint4 y = make_uint4(odd_half[0], odd_half[1], odd_half[2], odd_half[3]);
      uint4 *first = reinterpret_cast<uint4 *>(to + 4 * k), *second = reinterpret_cast<uint4 *>(to + 4 * k + kBlock * kSize);
      if constexpr (kBulk) __stcs(first, x), __stcs(second, y); // more than the L2 holds, as a rule: 2 us of 37
      else *first = x, *second = y;
    }
  }
}

bool power_of_two(float g) {
  int e;
  return std::frexp(g, &e) == 0.5f;
}

template <int D, int DT, bool kBulk, int U>
cudaError_t run_rows_u(const MxRowsArgs &a, bool write, cudaStream_t s) {
  constexpr int kRows = kThreads / (D / kBlock);
  const unsigned sides = a.x[0] && a.x[1] ? 2 : 1;
  int tshift = 0;
  dim3 grid;
  if (kBulk) {
    grid = dim3((a.T + U * kRows - 1) / (U * kRows), sides * a.c.Hkv, a.c.B);
  } else {
    while ((1 << tshift) < a.T) ++tshift;
    const long long heads = static_cast<long long>(a.c.B) * a.c.Hkv, per = kRows >> tshift;
    grid = dim3(static_cast<unsigned>((heads + per - 1) / per), 1, sides);
  }
  if (!write) return launch_pdl(mx_read_kernel<D, DT, kBulk, U>, grid, dim3(kThreads), 0, s, a, tshift);
  if constexpr (DT != TQ_F32)
    if ((!a.x[0] || power_of_two(a.c.g[0])) && (!a.x[1] || power_of_two(a.c.g[1])))
      return launch_pdl(mx_write_kernel<D, DT, kBulk, U, true>, grid, dim3(kThreads), 0, s, a, tshift);
  return launch_pdl(mx_write_kernel<D, DT, kBulk, U, false>, grid, dim3(kThreads), 0, s, a, tshift);
}

// Small calls have less than a CTA's rows of a head; bulk calls take four rows a thread where that leaves
// four CTAs for each SM, else two (read and write of 16 x 8 x 4096 rows of 128: 121 and 129 us; of 5 x
// 12 x 777 rows of 64: 8.8 and 7.2 us; one row a thread: 155 and 7.9 us).
template <int D, int DT>
cudaError_t run_rows(const MxRowsArgs &a, bool write, cudaStream_t s) {
  constexpr int kRows = kThreads / (D / kBlock);
  if (a.T <= kRows) return run_rows_u<D, DT, false, 1>(a, write, s);
  const long long ctas = static_cast<long long>(a.c.B) * a.c.Hkv * (a.x[0] && a.x[1] ? 2 : 1) * (a.T / (4 * kRows));
  return ctas >= 4 * 148 ? run_rows_u<D, DT, true, 4>(a, write, s) : run_rows_u<D, DT, true, 2>(a, write, s);
}

template <int D>
cudaError_t run_rows_d(const MxRowsArgs &a, bool write, cudaStream_t s) {
  if (a.dtype == TQ_F32) return run_rows<D, TQ_F32>(a, write, s);
  if (a.dtype == TQ_BF16) return run_rows<D, TQ_BF16>(a, write, s);
  return run_rows<D, TQ_F16>(a, write, s);
}

cudaError_t run_rows_any(const MxRowsArgs &a, bool write, cudaStream_t s) {
  if (a.c.d == 64) return run_rows_d<64>(a, write, s);
  if (a.c.d == 128) return run_rows_d<128>(a, write, s);
  return run_rows_d<256>(a, write, s);
}

} // namespace

cudaError_t launch_mx_write(const MxRowsArgs &a, cudaStream_t s) { return run_rows_any(a, true, s); }
cudaError_t launch_mx_read(const MxRowsArgs &a, cudaStream_t s) { return run_rows_any(a, false, s); }

} // namespace tq
