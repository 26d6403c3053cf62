// Write and read of the microscaled 4-bit paged cache.
//
// Write: a block of 16 elements x has the scale byte S = E4M3(min(max|x| / (6 g), 448)) and the
// codes E2M1(x / (S g)), both to nearest with ties to even; a NaN or infinity in the block makes
// S NaN (0x7F, codes 0), so that it stays visible. Read: E2M1 * S * g, one rounding in fp32 and
// one to the output's type.
//
// Both stream: a thread owns one block of one row (two 16-byte loads of 16-bit input, 9 bytes
// out), so a row's blocks and the rows of one head are contiguous across a warp, and nothing is
// kept between threads. They are bound by HBM (write: 2 + 9/16 bytes an element). Ties are
// common (16-bit inputs over a 4-bit scale hit an E2M1 midpoint about once in 64), so x / (S g)
// has to be the correctly rounded quotient: a product with the reciprocal alone lands on the
// wrong side of them. One reciprocal serves the block; each quotient is corrected by its exact
// remainder (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000",
// 1990), three FMA-pipe operations instead of a division.
#include "mx.cuh"

namespace tq {
namespace {

using namespace mx;

constexpr int kThreads = 256;

// Which (sequence, head, row, block) a thread owns: D/16 threads a row, `tt` consecutive rows of
// one head, then the next head or sequence. Small calls (one new token) fill CTAs with heads.
struct RowIndex {
  int b, h, t, blk;
  bool ok;
};

template <int D>
__device__ __forceinline__ RowIndex row_index(const MxRowsArgs &a, int tshift, int tchunks) {
  constexpr int kPer = D / kBlock, kRows = kThreads / kPer;
  const int r = threadIdx.x / kPer;
  const int chunk = blockIdx.x / tchunks;
  const int bh = chunk * (kRows >> tshift) + (r >> tshift);
  RowIndex i;
  i.blk = threadIdx.x % kPer;
  i.t = ((blockIdx.x - chunk * tchunks) << tshift) + (r & ((1 << tshift) - 1));
  i.b = bh / a.c.Hkv;
  i.h = bh - i.b * a.c.Hkv;
  i.ok = i.b < a.c.B && i.t < a.T;
  return i;
}

// Record index of row t of the batch, or -1 (not a row of the sequence, or not on a mapped page).
__device__ __forceinline__ long long record_of(const MxRowsArgs &a, const RowIndex &i) {
  const int n = clamp_count(a.counts, i.b, a.T);
  const long long pos = static_cast<long long>(__ldg(a.lens + i.b)) - n + i.t;
  if (i.t >= n || pos < 0 || (pos >> a.c.pshift) >= a.c.maxp) return -1;
  const int page = __ldg(a.c.bt + static_cast<long long>(i.b) * a.c.maxp + (pos >> a.c.pshift));
  if (page < 0 || page >= a.c.num_pages) return -1;
  return ((static_cast<long long>(page) * a.c.Hkv + i.h) << a.c.pshift) + (pos & ((1 << a.c.pshift) - 1));
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads) mx_write_kernel(const MxRowsArgs a, int tshift, int tchunks) {
  pdl_wait();
  const int which = a.x[0] && a.x[1] ? blockIdx.y : (a.x[0] ? 0 : 1);
  const RowIndex i = row_index<D>(a, tshift, tchunks);
  if (!i.ok) return;
  const long long rec = record_of(a, i);
  if (rec < 0) return;
  const long long *st = a.st[which];
  float v[kBlock];
  load_vec<kBlock>(a.x[which], DT, static_cast<size_t>(i.b * st[0] + i.h * st[1] + i.t * st[2] + i.blk * kBlock), v);
  float top = 0.0f;
  uint32_t bits = 0; // the largest |x| as bits: NaN and infinity compare above every finite value
#pragma unroll
  for (int k = 0; k < kBlock; ++k) bits = max(bits, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  top = __uint_as_float(bits);
  const float g = a.c.g[which];
  uint32_t s = 0x7Fu;
  uint2 codes = make_uint2(0u, 0u);
  if (bits < 0x7F800000u) {
    const float t = __fdiv_rn(top, 6.0f * g);
    s = float_to_e4m3(fminf(t, 448.0f));
    const float step = e4m3_to_float(s) * g;
    if (s != 0) {
      const float r = __frcp_rn(step);
      if (t > 448.0f) { // saturated: larger elements are 6 all the same; keeps the quotients finite
#pragma unroll
        for (int k = 0; k < kBlock; ++k) v[k] = fminf(fmaxf(v[k], -8.0f * step), 8.0f * step);
      }
#pragma unroll
      for (int k = 0; k < kBlock; ++k) {
        const float u = v[k] * r;
        v[k] = fmaf(fmaf(-u, step, v[k]), r, u);
      }
      codes.x = float_to_e2m1(v);
      codes.y = float_to_e2m1(v + 8);
    }
  }
  *reinterpret_cast<uint2 *>(a.c.codes[which] + rec * (D / 2) + i.blk * 8) = codes;
  a.c.scales[which][rec * (D / kBlock) + i.blk] = static_cast<uint8_t>(s);
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads) mx_read_kernel(const MxRowsArgs a, int tshift, int tchunks) {
  pdl_wait();
  const int which = a.x[0] && a.x[1] ? blockIdx.y : (a.x[0] ? 0 : 1);
  const RowIndex i = row_index<D>(a, tshift, tchunks);
  if (!i.ok) return;
  const long long rec = record_of(a, i);
  float v[kBlock];
#pragma unroll
  for (int k = 0; k < kBlock; ++k) v[k] = 0.0f;
  if (rec >= 0) {
    const uint2 codes = *reinterpret_cast<const uint2 *>(a.c.codes[which] + rec * (D / 2) + i.blk * 8);
    const float s = e4m3_to_float(a.c.scales[which][rec * (D / kBlock) + i.blk]);
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t h[4];
      e2m1_to_h2(w[k], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        v[8 * k + 2 * j] = f.x * s * a.c.g[which];
        v[8 * k + 2 * j + 1] = f.y * s * a.c.g[which];
      }
    }
  }
  const long long *st = a.st[which];
  store_vec<kBlock>(a.x[which], DT, static_cast<size_t>(i.b * st[0] + i.h * st[1] + i.t * st[2] + i.blk * kBlock), v);
}

template <int D, int DT>
cudaError_t run_rows(const MxRowsArgs &a, bool write, cudaStream_t s) {
  constexpr int kRows = kThreads / (D / kBlock);
  int tshift = 0;
  while ((1 << tshift) < a.T && (1 << tshift) < kRows) ++tshift;
  const int tchunks = (a.T + (1 << tshift) - 1) >> tshift;
  const long long heads = static_cast<long long>(a.c.B) * a.c.Hkv, per = kRows >> tshift;
  const dim3 grid(static_cast<unsigned>((heads + per - 1) / per * tchunks), a.x[0] && a.x[1] ? 2 : 1);
  return write ? launch_pdl(mx_write_kernel<D, DT>, grid, dim3(kThreads), 0, s, a, tshift, tchunks)
               : launch_pdl(mx_read_kernel<D, DT>, grid, dim3(kThreads), 0, s, a, tshift, tchunks);
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
