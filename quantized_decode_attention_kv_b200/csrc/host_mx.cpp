// C-ABI host layer of the microscaled 4-bit paged cache and of the page pools: argument
// validation and the calls into the CUDA launchers. Nothing here allocates device memory or
// synchronises.
#include "../../include/tq.h"
#include "tq_internal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <exception>
#include <vector>

namespace {

using tq::fail;

bool aligned(const void *p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int cuda_status(cudaError_t e, const char *what) {
  return e == cudaSuccess ? TQ_OK : fail(TQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The current device and its SM count, asked for once per device.
int current_device(int *dev, int *sms) {
  static std::atomic<int> known[64];
  if (cudaGetDevice(dev) != cudaSuccess) return fail(TQ_ERR_CUDA, "cannot query the current device");
  *sms = *dev < 64 ? known[*dev].load(std::memory_order_relaxed) : 0;
  if (*sms) return TQ_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return fail(TQ_ERR_CUDA, "cannot query the device's SM count");
  if (*dev < 64) known[*dev].store(*sms, std::memory_order_relaxed);
  return TQ_OK;
}

bool dtype_ok(int dt) { return dt == TQ_F32 || dt == TQ_BF16 || dt == TQ_F16; }

int page_shift(int page_size) {
  if (page_size < 16 || (page_size & (page_size - 1))) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

int check_mx(const tq_mx_cache *c, tq::MxCacheArgs *a) {
  if (!c) return fail(TQ_ERR_INVALID_ARG, "cache is NULL");
  if (c->B < 1 || c->Hkv < 1 || c->num_pages < 1 || c->max_pages < 1 || c->B > 65535 || c->Hkv > 4096)
    return fail(TQ_ERR_INVALID_ARG, "bad cache shape B=%d (1..65535) Hkv=%d (1..4096) num_pages=%d max_pages=%d",
                c->B, c->Hkv, c->num_pages, c->max_pages);
  if (c->d != 64 && c->d != 128 && c->d != 256)
    return fail(TQ_ERR_UNSUPPORTED, "d=%d: the microscaled cache holds head_dim 64, 128 or 256", c->d);
  const int shift = page_shift(c->page_size);
  if (shift < 0) return fail(TQ_ERR_INVALID_ARG, "page_size=%d must be a power of two >= 16", c->page_size);
  if (static_cast<long long>(c->max_pages) * c->page_size > (1ll << 30))
    return fail(TQ_ERR_INVALID_ARG, "max_pages=%d pages of %d positions pass 2^30", c->max_pages, c->page_size);
  // the attention kernel numbers 16-byte chunks of codes in 32 bits: 64 GiB an array
  if (static_cast<double>(c->num_pages) * c->Hkv * c->page_size * (c->d / 2) > 0x1p36)
    return fail(TQ_ERR_INVALID_ARG, "pool of %d pages x %d heads x %d positions of d=%d: codes pass 64 GiB",
                c->num_pages, c->Hkv, c->page_size, c->d);
  const float lo = 0x1p-64f, hi = 0x1p64f;
  if (!(c->k_scale >= lo && c->k_scale <= hi) || !(c->v_scale >= lo && c->v_scale <= hi))
    return fail(TQ_ERR_INVALID_ARG, "k_scale=%g and v_scale=%g must lie in 2^-64..2^64", c->k_scale, c->v_scale);
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16) ||
      !aligned(c->block_table, 16))
    return fail(TQ_ERR_INVALID_ARG, "codes, scales and block_table must be non-NULL and 16-byte aligned");
  *a = tq::MxCacheArgs{c->B, c->Hkv, c->d, shift, c->max_pages, c->num_pages, {c->k_scale, c->v_scale},
                       {c->k_codes, c->v_codes}, {c->k_scales, c->v_scales}, c->block_table};
  return TQ_OK;
}

// Strides of one input tensor: given (checked) or those of a contiguous [B][Hkv][T][d].
int take_strides(const int64_t *given, const tq_mx_cache &c, int T, int dtype, const char *name, long long (&st)[3]) {
  const int per16 = dtype == TQ_F32 ? 4 : 8;
  st[0] = static_cast<long long>(c.Hkv) * T * c.d;
  st[1] = static_cast<long long>(T) * c.d;
  st[2] = c.d;
  for (int i = 0; given && i < 3; ++i) {
    if (given[i] < 0 || given[i] % per16 || given[i] > (1ll << 46))
      return fail(TQ_ERR_INVALID_ARG, "%s stride %lld must be >= 0 and a multiple of 16 bytes", name,
                  static_cast<long long>(given[i]));
    st[i] = given[i];
  }
  return TQ_OK;
}

int check_rows(const void *K, const void *V, int dtype, int T, const int32_t *lens, const int32_t *counts,
               const tq_mx_cache *cache, tq::MxRowsArgs *a) {
  int st = check_mx(cache, &a->c);
  if (st) return st;
  if (!dtype_ok(dtype)) return fail(TQ_ERR_INVALID_ARG, "dtype=%d is not F32/BF16/F16", dtype);
  if (!K && !V && T != 0) return fail(TQ_ERR_INVALID_ARG, "K and V are both NULL"); // without rows both may be
  if ((K && !aligned(K, 16)) || (V && !aligned(V, 16)))
    return fail(TQ_ERR_INVALID_ARG, "K/V pointers must be 16-byte aligned");
  if (T < 0 || T > (1 << 30)) return fail(TQ_ERR_INVALID_ARG, "T=%d must be in 0..2^30", T);
  if (static_cast<double>(cache->B) * cache->Hkv * T * (cache->d / 16) >= 128.0 * 2147483647.0)
    return fail(TQ_ERR_INVALID_ARG, "B=%d x Hkv=%d x T=%d rows are too many for one call", cache->B, cache->Hkv, T);
  if (!aligned(lens, 4) || (counts && !aligned(counts, 4)))
    return fail(TQ_ERR_INVALID_ARG, "lens must be non-NULL, lens and counts 4-byte aligned");
  a->x[0] = const_cast<void *>(K);
  a->x[1] = const_cast<void *>(V);
  for (int i = 0; i < 2; ++i) a->inv6g[i] = 1.0f / (6.0f * a->c.g[i]);
  a->dtype = dtype;
  a->T = T;
  a->lens = lens;
  a->counts = counts;
  return TQ_OK;
}

int check_decode_shape(int Hq, int Lq, const tq_mx_cache *cache, tq::MxDecodeArgs *a) {
  int st = check_mx(cache, &a->c);
  if (st) return st;
  if (Hq < 1 || Hq % cache->Hkv || Hq > 65535)
    return fail(TQ_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d (<= 65535)", Hq, cache->Hkv);
  if (Lq < 1 || Lq > 16) return fail(TQ_ERR_INVALID_ARG, "Lq=%d: must be 1..16 queries a sequence", Lq);
  // the kernel numbers 16-position tiles over all sequences and row blocks (of 8 rows at least) in 32 bits
  const double blocks = std::ceil(static_cast<double>(Lq) * (Hq / cache->Hkv) / 8);
  const double tiles = static_cast<double>(cache->max_pages) * (cache->page_size / 16) + 4;
  if (cache->B * blocks * cache->Hkv * tiles >= 4294967296.0)
    return fail(TQ_ERR_INVALID_ARG, "B=%d x Hkv=%d x %d positions are too many for one call", cache->B, cache->Hkv,
                cache->max_pages * cache->page_size);
  int dev = 0, sms = 0;
  st = current_device(&dev, &sms);
  if (st) return st;
  a->Hq = Hq;
  a->Lq = Lq;
  a->plan = tq::plan_mx_decode(cache->Hkv, cache->d, Hq, Lq, dev, sms);
  return TQ_OK;
}

int check_pool(const tq_page_pool *p) {
  if (!p) return fail(TQ_ERR_INVALID_ARG, "pool is NULL");
  if (p->B < 1 || p->B > tq::kMaxPoolB || p->max_pages < 1 || p->num_pages < 1 || p->num_pages > (1 << 30))
    return fail(TQ_ERR_INVALID_ARG, "bad pool shape B=%d (1..%d) max_pages=%d num_pages=%d", p->B, tq::kMaxPoolB,
                p->max_pages, p->num_pages);
  if (page_shift(p->page_size) < 0)
    return fail(TQ_ERR_INVALID_ARG, "page_size=%d must be a power of two >= 16", p->page_size);
  if (static_cast<long long>(p->max_pages) * p->page_size > (1ll << 30))
    return fail(TQ_ERR_INVALID_ARG, "max_pages=%d pages of %d positions pass 2^30", p->max_pages, p->page_size);
  if (!aligned(p->refs, 16) || !aligned(p->block_table, 16) || !aligned(p->lens, 16))
    return fail(TQ_ERR_INVALID_ARG, "refs, block_table and lens must be non-NULL and 16-byte aligned");
  return TQ_OK;
}

int check_arrays(const tq_page_array *arrays, int n, int least) {
  if (n < least || n > tq::kMaxPageArrays || (n > 0 && !arrays))
    return fail(TQ_ERR_INVALID_ARG, "n_arrays=%d must be %d..%d, arrays non-NULL", n, least, tq::kMaxPageArrays);
  for (int i = 0; i < n; ++i)
    if (!aligned(arrays[i].base, 16) || arrays[i].page_bytes == 0 || arrays[i].page_bytes % 16 ||
        arrays[i].page_bytes >= (1ull << 31))
      return fail(TQ_ERR_INVALID_ARG, "arrays[%d]: base must be 16-byte aligned and page_bytes=%zu a multiple of 16 "
                  "below 2^31", i, arrays[i].page_bytes);
  return TQ_OK;
}

int check_workspace(const void *ws, size_t have, size_t need) {
  if (!aligned(ws, 16) || have < need)
    return fail(TQ_ERR_WORKSPACE, "workspace needs %zu bytes (16-byte aligned), got %zu", need, ws ? have : 0);
  return TQ_OK;
}

} // namespace

extern "C" {

int tq_quantize_kv_mx(const void *K, const void *V, int dtype, int T, const int64_t *k_strides,
                      const int64_t *v_strides, const int32_t *lens, const int32_t *counts,
                      const tq_mx_cache *cache, void *stream) {
  tq::MxRowsArgs a{};
  int st = check_rows(K, V, dtype, T, lens, counts, cache, &a);
  if (st) return st;
  st = take_strides(k_strides, *cache, T, dtype, "K", a.st[0]);
  if (st) return st;
  st = take_strides(v_strides, *cache, T, dtype, "V", a.st[1]);
  if (st) return st;
  if (T == 0) return TQ_OK;
  return cuda_status(tq::launch_mx_write(a, static_cast<cudaStream_t>(stream)), "microscaled write launch");
}

int tq_dequantize_mx(const tq_mx_cache *cache, int T, const int32_t *lens, const int32_t *counts, void *K,
                     void *V, int dtype, void *stream) {
  tq::MxRowsArgs a{};
  int st = check_rows(K, V, dtype, T, lens, counts, cache, &a);
  if (st) return st;
  for (int i = 0; i < 2; ++i) take_strides(nullptr, *cache, T, dtype, "", a.st[i]);
  if (T == 0) return TQ_OK;
  return cuda_status(tq::launch_mx_read(a, static_cast<cudaStream_t>(stream)), "microscaled read launch");
}

size_t tq_decode_mx_workspace_bytes(int Hq, int Lq, const tq_mx_cache *cache) {
  tq::MxDecodeArgs a{};
  return check_decode_shape(Hq, Lq, cache, &a) ? 0 : a.plan.ws_bytes;
}

int tq_decode_attention_mx(const void *q, int dtype, int Hq, int Lq, const int32_t *lens, const int32_t *counts,
                           float scale, const tq_mx_cache *cache, void *out, int out_dtype, void *ws,
                           size_t ws_bytes, void *stream) {
  if (dtype != TQ_BF16 && dtype != TQ_F16)
    return dtype_ok(dtype) ? fail(TQ_ERR_UNSUPPORTED, "queries must be BF16 or F16")
                           : fail(TQ_ERR_INVALID_ARG, "dtype=%d is not BF16/F16", dtype);
  if (!dtype_ok(out_dtype)) return fail(TQ_ERR_INVALID_ARG, "out_dtype=%d is not F32/BF16/F16", out_dtype);
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(TQ_ERR_INVALID_ARG, "q/out must be non-NULL and 16-byte aligned");
  if (!aligned(lens, 4) || (counts && !aligned(counts, 4)))
    return fail(TQ_ERR_INVALID_ARG, "lens must be non-NULL, lens and counts 4-byte aligned");
  if (!std::isfinite(scale)) return fail(TQ_ERR_INVALID_ARG, "scale is not finite");
  tq::MxDecodeArgs a{};
  int st = check_decode_shape(Hq, Lq, cache, &a);
  if (st) return st;
  st = check_workspace(ws, ws_bytes, a.plan.ws_bytes);
  if (st) return st;
  a.q = q;
  a.dtype = dtype;
  a.out_dtype = out_dtype;
  a.lens = lens;
  a.counts = counts;
  a.scale = scale;
  a.out = out;
  a.ws = ws;
  return cuda_status(tq::launch_mx_decode(a, static_cast<cudaStream_t>(stream)), "microscaled decode launch");
}

int tq_paged_cache_arrays(const tq_paged_cache *c, tq_page_array *out) {
  if (!c || !out || c->Hkv < 1 || page_shift(c->page_size) < 0) {
    fail(TQ_ERR_INVALID_ARG, "cache or out is NULL, or the cache's shape is bad");
    return 0;
  }
  const size_t rows = static_cast<size_t>(c->Hkv) * c->page_size;
  const tq_qcfg cfg[2] = {c->kc, c->vc};
  void *const codes[2] = {c->k_codes, c->v_codes}, *const norm[2] = {c->k_norm, c->v_norm};
  void *const signs[2] = {c->k_signs, c->v_signs}, *const rnorm[2] = {c->k_rnorm, c->v_rnorm};
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (tq_record_bytes(c->d, cfg[i]) == 0) return 0;
    const size_t cb = tq_code_bytes(c->d, cfg[i]), sb = tq_sign_bytes(c->d, cfg[i]);
    if (cb) out[n++] = {codes[i], rows * cb};
    out[n++] = {norm[i], rows * 2};
    if (sb) {
      out[n++] = {signs[i], rows * sb};
      out[n++] = {rnorm[i], rows * 2};
    }
  }
  return check_arrays(out, n, 1) ? 0 : n;
}

int tq_mx_cache_arrays(const tq_mx_cache *c, tq_page_array *out) {
  tq::MxCacheArgs a{};
  if (!out) {
    fail(TQ_ERR_INVALID_ARG, "out is NULL");
    return 0;
  }
  if (check_mx(c, &a)) return 0;
  const size_t rows = static_cast<size_t>(c->Hkv) * c->page_size;
  for (int i = 0; i < 2; ++i) {
    out[2 * i] = {a.codes[i], rows * (c->d / 2)};
    out[2 * i + 1] = {a.scales[i], rows * (c->d / 16)};
  }
  return check_arrays(out, 4, 1) ? 0 : 4;
}

size_t tq_pages_workspace_bytes(const tq_page_pool *pool) {
  return check_pool(pool) ? 0 : tq::pages_workspace_bytes(*pool);
}

int tq_pages_extend(const tq_page_pool *pool, const int32_t *need, int32_t *status, void *stream) {
  int st = check_pool(pool);
  if (st) return st;
  if (!aligned(need, 4) || !aligned(status, 4))
    return fail(TQ_ERR_INVALID_ARG, "need/status must be non-NULL and 4-byte aligned");
  return cuda_status(tq::launch_pages_extend(*pool, need, nullptr, status, static_cast<cudaStream_t>(stream)),
                     "page extend launch");
}

int tq_pages_extend_granted(const tq_page_pool *pool, const int32_t *need, int32_t *granted, int32_t *status,
                            void *stream) {
  int st = check_pool(pool);
  if (st) return st;
  if (!aligned(need, 4) || !aligned(granted, 4) || !aligned(status, 4))
    return fail(TQ_ERR_INVALID_ARG, "need/granted/status must be non-NULL and 4-byte aligned");
  return cuda_status(tq::launch_pages_extend(*pool, need, granted, status, static_cast<cudaStream_t>(stream)),
                     "page extend launch");
}

int tq_pages_fork(const tq_page_pool *pool, const tq_page_array *arrays, int n_arrays,
                  const int32_t *parent_of, int32_t *status, void *ws, size_t ws_bytes, void *stream) {
  int st = check_pool(pool);
  if (st) return st;
  st = check_arrays(arrays, n_arrays, 0);
  if (st) return st;
  if (!aligned(parent_of, 4) || !aligned(status, 4))
    return fail(TQ_ERR_INVALID_ARG, "parent_of/status must be non-NULL and 4-byte aligned");
  st = check_workspace(ws, ws_bytes, tq::pages_workspace_bytes(*pool));
  if (st) return st;
  int dev = 0, sms = 0;
  st = current_device(&dev, &sms);
  if (st) return st;
  return cuda_status(tq::launch_pages_fork(*pool, arrays, n_arrays, parent_of, status, ws, sms,
                                           static_cast<cudaStream_t>(stream)), "page fork launch");
}

int tq_pages_free(const tq_page_pool *pool, const int32_t *leaving, void *stream) {
  int st = check_pool(pool);
  if (st) return st;
  if (!aligned(leaving, 4)) return fail(TQ_ERR_INVALID_ARG, "leaving must be non-NULL and 4-byte aligned");
  return cuda_status(tq::launch_pages_free(*pool, leaving, static_cast<cudaStream_t>(stream)), "page free launch");
}

int tq_pages_compact(const tq_page_pool *pool, const tq_page_array *arrays, int n_arrays, int32_t *live,
                     void *ws, size_t ws_bytes, void *stream) {
  int st = check_pool(pool);
  if (st) return st;
  st = check_arrays(arrays, n_arrays, 0);
  if (st) return st;
  if (!aligned(live, 4)) return fail(TQ_ERR_INVALID_ARG, "live must be non-NULL and 4-byte aligned");
  st = check_workspace(ws, ws_bytes, tq::pages_workspace_bytes(*pool));
  if (st) return st;
  int dev = 0, sms = 0;
  st = current_device(&dev, &sms);
  if (st) return st;
  return cuda_status(tq::launch_pages_compact(*pool, arrays, n_arrays, live, ws, sms,
                                              static_cast<cudaStream_t>(stream)), "page compact launch");
}

int tq_pages_copy(const tq_page_array *arrays, int n_arrays, int num_pages, const int *src, const int *dst,
                  int n, void *stream) {
  int st = check_arrays(arrays, n_arrays, 1);
  if (st) return st;
  if (num_pages < 1 || n < 0 || (n > 0 && (!src || !dst)))
    return fail(TQ_ERR_INVALID_ARG, "num_pages=%d, n=%d: need num_pages >= 1, n >= 0, src and dst", num_pages, n);
  if (n == 0) return TQ_OK;
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages)
      return fail(TQ_ERR_INVALID_ARG, "pair %d: pages %d -> %d outside 0..%d", i, src[i], dst[i], num_pages - 1);
  try {
    std::vector<int> to(dst, dst + n);
    std::sort(to.begin(), to.end());
    const auto twice = std::adjacent_find(to.begin(), to.end());
    if (twice != to.end()) return fail(TQ_ERR_INVALID_ARG, "page %d is the destination of two copies", *twice);
    for (int i = 0; i < n; ++i)
      if (std::binary_search(to.begin(), to.end(), src[i]))
        return fail(TQ_ERR_INVALID_ARG, "page %d is a source and a destination", src[i]);
  } catch (const std::exception &) {
    return fail(TQ_ERR_INVALID_ARG, "out of host memory for %d pairs", n);
  }
  int dev = 0, sms = 0;
  st = current_device(&dev, &sms);
  if (st) return st;
  return cuda_status(tq::launch_pages_copy(arrays, n_arrays, src, dst, n, sms, static_cast<cudaStream_t>(stream)),
                     "page copy launch");
}

} // extern "C"
