"""GPU tests of the microscaled 4-bit paged cache (write, read back, attention) against the float64
oracle, through the Python binding of the C ABI."""
import math

import numpy as np
import pytest
import torch

from oracle import mx_oracle as M

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the GPU tier always has a device
    pytest.skip("needs a CUDA device", allow_module_level=True)

from quantized_decode_attention_kv_b200 import tq  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(B, max_pages, num_pages, seed):
    perm = np.random.default_rng(seed).permutation(num_pages)[: B * max_pages]
    return torch.from_numpy(perm.reshape(B, max_pages).astype(np.int32)).cuda()


def _cache(B, Hkv, d, page, max_pages, spare=3, g=(1.0, 1.0), seed=0):
    num_pages = B * max_pages + spare
    return tq.TQMXCache(B, Hkv, d, page, num_pages, max_pages, _table(B, max_pages, num_pages, seed), *g)


def _np(x):
    return x.detach().cpu().double().numpy()


def _randn(shape, dtype, seed, loud=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if loud:
        x[..., :3] *= 20.0
        x *= torch.rand(*shape[:-1], 1, generator=g) * 1.5 + 0.5
    return x.to(dtype)


def _records(cache, side, b, h, pos):
    """Code and scale bytes of positions pos of (b, h), through the block table."""
    pos = torch.as_tensor(pos)
    pages = cache.block_table[b].cpu()[pos // cache.page_size].long()
    slot = pos % cache.page_size
    return (cache[f"{side}_codes"].cpu()[pages, h, slot].numpy(), cache[f"{side}_scales"].cpu()[pages, h, slot].numpy())


def _fill(cache, byte):
    for t in cache.tensors.values():
        t.fill_(byte)


def _touched(cache, side, lens, counts):
    """Mask [num_pages, page] of the slots the rows belong to."""
    m = np.zeros((cache.num_pages, cache.page_size), bool)
    bt = cache.block_table.cpu().numpy()
    for b, (L, n) in enumerate(zip(lens, counts)):
        for pos in range(max(L - n, 0), L):
            if pos < cache.max_pages * cache.page_size and 0 <= bt[b, pos // cache.page_size] < cache.num_pages:
                m[bt[b, pos // cache.page_size], pos % cache.page_size] = True
    return m


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("d,dtype,page,Hkv,T,hist,ragged,g", [
    (128, "bf16", 64, 8, 1, 130, False, 1.0),
    (128, "bf16", 16, 3, 77, 5, True, 0.25),
    (64, "f16", 32, 12, 33, 0, True, 2.0),
    (256, "f32", 16, 1, 50, 31, False, 1.0),
    (64, "f32", 128, 5, 1, 0, False, 0.37),   # a scale that is no power of two: float32 quotients
    (256, "bf16", 64, 2, 9, 200, True, 1.7e-3),
    (128, "f16", 16, 1, 600, 0, True, 1.0),
])
def test_write_matches_oracle_byte_for_byte(d, dtype, page, Hkv, T, hist, ragged, g):
    B = 4
    counts = [T, max(T // 3, 0), 0, T] if ragged else [T] * B
    lens = [hist + n + 2 * b for b, n in enumerate(counts)]
    K, V = _randn((B, Hkv, T, d), DT[dtype], 1), _randn((B, Hkv, T, d), DT[dtype], 2, loud=False)
    cache = _cache(B, Hkv, d, page, -(-max(lens) // page) + 1, g=(g, 2 * g))
    _fill(cache, 0xA5)
    tq.tq_quantize_kv_mx(K.cuda(), V.cuda(), cache, _i32(lens), _i32(counts) if ragged else None)
    torch.cuda.synchronize()
    wide = np.float64 if math.log2(g).is_integer() else np.float32
    for side, x, gg in (("k", K, g), ("v", V, 2 * g)):
        for b in range(B):
            for h in range(Hkv):
                n = counts[b]
                codes, s = M.quantise(_np(x[b, h, :n]), np.float32(gg), wide)
                got_c, got_s = _records(cache, side, b, h, np.arange(lens[b] - n, lens[b]))
                np.testing.assert_array_equal(got_s, s)
                # -0 and 0 stand for one value: compare the values the codes stand for
                np.testing.assert_array_equal(M.values(got_c, s, gg), M.values(M.pack(codes), s, gg))
        seen = _touched(cache, side, lens, counts)
        for key in ("codes", "scales"):  # every other record is as it was
            pool = cache[f"{side}_{key}"].cpu().numpy()
            assert (pool.transpose(0, 2, 1, 3)[~seen] == 0xA5).all()
    # and back: every row of the batch, in every type
    for out_t in DT.values():
        Ko, Vo = (torch.full((B, Hkv, T, d), 7.0, dtype=out_t, device="cuda") for _ in range(2))
        tq.tq_dequantize_mx(cache, _i32(lens), Ko, Vo, _i32(counts) if ragged else None)
        for side, out, gg in (("k", Ko, g), ("v", Vo, 2 * g)):
            for b in range(B):
                n = counts[b]
                assert (out[b, :, n:] == 0).all()
                for h in range(Hkv):
                    rec = _records(cache, side, b, h, np.arange(lens[b] - n, lens[b]))
                    # E2M1 * S is exact in float32; the product with the scale is rounded there, once
                    want = torch.from_numpy(M.values(*rec, 1.0).astype(np.float32) * np.float32(gg)).to(out_t)
                    assert torch.equal(out[b, h, :n].cpu(), want)


def test_write_takes_the_slices_of_a_fused_projection():
    B, T, Hq, Hkv, d = 3, 21, 4, 2, 128
    x = _randn((B, T, Hq + 2 * Hkv, d), torch.bfloat16, 3).cuda()
    K, V = x[:, :, Hq:Hq + Hkv].transpose(1, 2), x[:, :, Hq + Hkv:].transpose(1, 2)
    assert not K.is_contiguous()
    a, b = _cache(B, Hkv, d, 16, 2), _cache(B, Hkv, d, 16, 2)
    lens = _i32([T] * B)
    tq.tq_quantize_kv_mx(K, V, a, lens)
    tq.tq_quantize_kv_mx(K.contiguous(), V.contiguous(), b, lens)
    one = K[:, :1].expand(B, Hkv, T, d)  # a broadcast head: stride 0
    c, e = _cache(B, Hkv, d, 16, 2), _cache(B, Hkv, d, 16, 2)
    tq.tq_quantize_kv_mx(one, None, c, lens)
    tq.tq_quantize_kv_mx(one.contiguous(), None, e, lens)
    for key in a.tensors:
        assert torch.equal(a[key], b[key]) and torch.equal(c[key], e[key])
    assert (c["v_codes"] == 0).all()  # V was None


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -7, 0.75])  # 0.75: not a power of two, S g still exact in fp32
def test_every_16_bit_value_at_every_scale_rounds_right(dtype, g):
    # blocks of fifteen values and one that sets the scale to S = 1 + m / 8: all finite patterns up to it,
    # of both signs
    t = DT[dtype]
    every = torch.arange(0x7C00 if dtype == "f16" else 0x7F80, dtype=torch.int32).to(torch.int16).view(t).double()
    rows = []
    for m in range(8):
        top = 6.0 * (1 + m / 8) * g
        assert float(torch.tensor(top, dtype=t)) == top
        v = every[(every <= top) & (every >= top / 4096)]  # smaller ones are far below the first midpoint
        v = torch.cat([v, -v, torch.zeros(-2 * len(v) % 15, dtype=torch.float64)]).view(-1, 15)
        rows.append(torch.cat([v, torch.full((len(v), 1), top, dtype=torch.float64)], dim=1))
    x = torch.cat(rows)
    x = torch.cat([x, torch.zeros(-len(x) % 4, 16, dtype=torch.float64)]).view(1, 1, -1, 64).to(t)
    T = x.shape[2]
    cache = _cache(1, 1, 64, 64, -(-T // 64), g=(g, g))
    tq.tq_quantize_kv_mx(x.cuda(), None, cache, _i32([T]))
    codes, s = M.quantise(_np(x[0, 0]), g)
    got_c, got_s = _records(cache, "k", 0, 0, np.arange(T))
    np.testing.assert_array_equal(got_s, s)
    np.testing.assert_array_equal(M.values(got_c, s, g), M.values(M.pack(codes), s, g))


@pytest.mark.parametrize("d,dtype,B,Hkv,T,page,layout", [
    (128, "bf16", 2, 3, 200, 16, "heads"),     # two rows a thread
    (128, "f16", 8, 8, 641, 64, "rows"),       # four rows a thread, ragged end
    (64, "f32", 8, 8, 1300, 32, "heads"),
    (256, "bf16", 8, 8, 330, 16, "rows"),
    (64, "f16", 1, 1, 129, 128, "rows"),
])
def test_bulk_calls_equal_calls_of_few_rows(d, dtype, B, Hkv, T, page, layout):
    """Whole prompts at once, from both layouts, one side or both: the bytes of calls of 16 rows each
    (which the oracle's tests cover), and the same rows back."""
    g = torch.Generator(device="cuda").manual_seed(T)
    shape = (B, T, Hkv, d) if layout == "heads" else (B, Hkv, T, d)
    K, V = (torch.randn(shape, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    if layout == "heads":  # a model's [sequence][row][head] layout
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    counts = [T] + [T - 1 - (37 * b) % T for b in range(1, B)]
    lens = [n + 5 * b for b, n in enumerate(counts)]
    max_pages = -(-max(lens) // page)
    a, b_, c = (_cache(B, Hkv, d, page, max_pages, g=(0.5, 2.0), seed=T) for _ in range(3))
    for cache in (a, b_, c):
        _fill(cache, 0x3C)
    tq.tq_quantize_kv_mx(K, V, a, _i32(lens), _i32(counts))
    tq.tq_quantize_kv_mx(K, None, b_, _i32(lens), _i32(counts))
    tq.tq_quantize_kv_mx(None, V, b_, _i32(lens), _i32(counts))
    for t in range(0, T, 16):
        n = min(16, T - t)
        now = [min(max(k - t, 0), n) for k in counts]
        tq.tq_quantize_kv_mx(K[:, :, t:t + n], V[:, :, t:t + n], c, _i32([L - k + t + m for L, k, m in zip(lens, counts, now)]),
                             _i32(now))
    for key in a.tensors:
        assert torch.equal(a[key], c[key]) and torch.equal(b_[key], c[key])
    for out_t in DT.values():
        big, few = ([torch.full((B, Hkv, T, d), 9.0, dtype=out_t, device="cuda") for _ in range(2)] for _ in range(2))
        tq.tq_dequantize_mx(a, _i32(lens), *big, _i32(counts))
        only = torch.full_like(big[1], 9.0)
        tq.tq_dequantize_mx(a, _i32(lens), None, only, _i32(counts))
        assert torch.equal(only, big[1])
        for t in range(0, T, 16):
            n = min(16, T - t)
            now = [min(max(k - t, 0), n) for k in counts]
            part = [torch.empty((B, Hkv, n, d), dtype=out_t, device="cuda") for _ in range(2)]
            tq.tq_dequantize_mx(a, _i32([L - k + t + m for L, k, m in zip(lens, counts, now)]), *part, _i32(now))
            for f, p in zip(few, part):
                f[:, :, t:t + n] = p
        assert all(torch.equal(x, y) for x, y in zip(big, few))


def test_strides_of_single_rows_and_sequences_do_not_matter():
    cache, other = _cache(1, 2, 64, 16, 2), _cache(1, 2, 64, 16, 2)
    base = _randn((2 * 64 + 7 + 3 * 64,), torch.bfloat16, 77).cuda()
    x = base.as_strided((1, 2, 1, 64), (7, 128, 3, 1))  # strides of size-1 dimensions that are no multiples of 16 bytes
    tq.tq_quantize_kv_mx(x, x, cache, _i32([5]))
    tq.tq_quantize_kv_mx(x.contiguous(), x.contiguous(), other, _i32([5]))
    for key in cache.tensors:
        assert torch.equal(cache[key], other[key])


@pytest.mark.parametrize("dtype", list(DT))
def test_write_of_special_values(dtype):
    t = DT[dtype]
    rows = torch.zeros(12, 64)
    rows[0] = 0.0
    rows[1, 5], rows[1, 20] = float("nan"), 1.0
    rows[2, 40], rows[2, 1] = float("-inf"), 3.0
    rows[3] = 6e4                              # above 6 * 448: saturates
    rows[3, 7], rows[3, 8], rows[3, 9] = -6e4, 2688.0, 100.0
    rows[4] = 2.0 ** -14                       # top / 6 rounds to the scale 0
    rows[4, 16] = 6 * 2.0 ** -9                # the smallest scale
    rows[4, 17] = -2.0 ** -9
    rows[5, :16] = torch.tensor([6, 0.25, -0.25, 0.75, -0.75, 1.25, 1.75, 2.5, -2.5, 3.5, 5, -5, 0.5, 4, -3, 1.5])
    rows[6, :16] = rows[5, :16] * 1.5          # ties at a scale that is no power of two
    rows[7] = -0.0
    rows[8] = torch.finfo(t).max
    rows[9] = torch.finfo(t).smallest_normal
    rows[10, ::2], rows[10, 1::2] = 1e-5, 4.0
    rows[11] = torch.linspace(-7, 7, 64)
    x = rows.to(t).reshape(1, 1, 12, 64).cuda()
    cache = _cache(1, 1, 64, 16, 1)
    tq.tq_quantize_kv_mx(x, x, cache, _i32([12]))
    with np.errstate(over="ignore"):
        codes, s = M.quantise(_np(x[0, 0]), 1.0)
    got_c, got_s = _records(cache, "k", 0, 0, np.arange(12))
    np.testing.assert_array_equal(got_s, s)
    np.testing.assert_array_equal(M.values(got_c, s, 1.0), M.values(M.pack(codes), s, 1.0))
    out = torch.empty_like(x, dtype=torch.float32)
    tq.tq_dequantize_mx(cache, _i32([12]), None, out)
    np.testing.assert_array_equal(_np(out[0, 0]), M.values(got_c, s, 1.0))
    assert torch.isnan(out[0, 0, 1, :16]).all() and (out[0, 0, 1, 20] > 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("g", [2.0 ** -64, 1.3 * 2.0 ** -63, 2.0 ** 64])
def test_values_far_above_and_below_the_scale(dtype, g):
    # top / (6 g) passes fp32 (saturates: every larger element is 6, signs stay), or is far below 2^-10 (zeros)
    t = DT[dtype]
    x = torch.zeros(1, 1, 3, 64)
    x[0, 0, 0], x[0, 0, 0, ::3] = torch.finfo(t).max, -torch.finfo(t).max
    x[0, 0, 1, :4] = torch.tensor([1.0, -1e4, 3e4, -torch.finfo(t).max])
    x[0, 0, 2] = torch.finfo(t).smallest_normal
    x = x.to(t).cuda()
    cache = _cache(1, 1, 64, 16, 1, g=(g, g))
    tq.tq_quantize_kv_mx(x, x, cache, _i32([3]))
    codes, s = M.quantise(_np(x[0, 0]), np.float32(g), np.float64)
    for side in "kv":
        got_c, got_s = _records(cache, side, 0, 0, np.arange(3))
        np.testing.assert_array_equal(got_s, s)
        np.testing.assert_array_equal(M.values(got_c, s, 1.0), M.values(M.pack(codes), s, 1.0))


def test_write_and_read_leave_out_what_has_no_place():
    B, Hkv, d, page = 5, 2, 64, 16
    cache = _cache(B, Hkv, d, page, 3)
    bt = cache.block_table
    bt[1, 1] = -1                      # unmapped
    bt[2, 0] = cache.num_pages         # no such page
    _fill(cache, 0x11)
    lens, counts = [20, 40, 20, 3, 60], [20, 20, 20, 9, 20]  # row 3: starts before 0; row 4: ends past the capacity
    x = _randn((B, Hkv, 20, d), torch.float16, 4).cuda()
    tq.tq_quantize_kv_mx(x, x, cache, _i32(lens), _i32(counts))
    out = torch.full((B, Hkv, 20, d), 9.0, dtype=torch.float32, device="cuda")
    tq.tq_dequantize_mx(cache, _i32(lens), out, None, _i32(counts))
    seen = _touched(cache, "k", lens, counts)
    assert (cache["k_codes"].cpu().numpy().transpose(0, 2, 1, 3)[~seen] == 0x11).all()
    tab = bt.cpu().numpy()
    for b in range(B):
        for t in range(20):
            pos = lens[b] - counts[b] + t
            here = t < counts[b] and 0 <= pos < 48 and 0 <= tab[b, pos // 16] < cache.num_pages
            if here:
                codes, s = M.quantise(_np(x[b, 1, t]), 1.0)
                np.testing.assert_array_equal(_np(out[b, 1, t]), M.values(M.pack(codes), s, 1.0))
            else:
                assert (out[b, :, t] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_calls_of_no_rows_do_nothing(dtype):
    cache = _cache(2, 2, 128, 16, 2)
    _fill(cache, 0x5A)
    x = torch.empty(2, 2, 0, 128, dtype=DT[dtype], device="cuda")
    for K, V in ((x, x), (x, None), (None, x)):
        for counts in (None, _i32([0, 0]), _i32([5, 0])):
            tq.tq_quantize_kv_mx(K, V, cache, _i32([7, 0]), counts)
            tq.tq_dequantize_mx(cache, _i32([7, 0]), K, V, counts)
    torch.cuda.synchronize()
    assert all((t == 0x5A).all() for t in cache.tensors.values())
    with pytest.raises(tq.TQError):
        tq.tq_quantize_kv_mx(None, None, cache, _i32([7, 0]))


# ------------------------------------------------------------------ attention
def _bound(att, d, T, out_dtype):
    """Largest admissible |error|, elementwise. Weights are fp16 (relative 2^-11; those below 2^-25 of
    the largest are off by at most 2^-36 of it, T of them on values up to att.v), scores are sums of d exact products in fp32 (each
    addition off by at most 2^-23, truncation included) scaled and shifted in log2 units (two
    roundings of 2^-24 of at most 1.4427 m each, a factor ln 2 back), ex2 is off by 2^-21, output
    sums of T products and the merges of the partials by 2^-23 an addition; numerator and
    denominator share the weights, so an error e of them costs e (a + |o|)."""
    e = 2.0 ** -11 + att.m * (d + 4) * 2.0 ** -23 + 2.0 ** -21 + (T + 64) * 2.0 ** -23
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}[out_dtype]
    return (att.a + np.abs(att.o)) * e * 1.01 + np.abs(att.o) * torch.finfo(out_dtype).eps / 2 * 1.01 + (
        T * 2.0 ** -36 * att.v + tiny)


def _setup(B, Hkv, d, page, lens, seed=0, g=(1.0, 1.0), spare=3, k_gain=0.3):
    """A cache filled to capacity with quantised rows (the tail pages hold rows of no sequence)."""
    max_pages = max(1, -(-max(lens) // page)) if isinstance(lens, list) else lens
    cache = _cache(B, Hkv, d, page, max_pages, spare, g, seed)
    T = max_pages * page
    K = (_randn((B, Hkv, T, d), torch.float32, seed + 10) * k_gain).to(torch.bfloat16).cuda()
    V = _randn((B, Hkv, T, d), torch.bfloat16, seed + 11, loud=False).cuda()
    tq.tq_quantize_kv_mx(K, V, cache, _i32([T] * B))
    return cache


def _dense(cache):
    """Values [B, Hkv, T, d] of keys and values in float64 by the oracle, and the mapped positions."""
    T = cache.max_pages * cache.page_size
    bt = cache.block_table.cpu().numpy()
    mapped = np.repeat((bt >= 0) & (bt < cache.num_pages), cache.page_size, axis=1)
    pages = np.where((bt >= 0) & (bt < cache.num_pages), bt, 0)
    out = []
    for side, g in (("k", cache.k_scale), ("v", cache.v_scale)):
        with np.errstate(invalid="ignore"):
            v = M.values(cache[f"{side}_codes"].cpu().numpy(), cache[f"{side}_scales"].cpu().numpy(), g)
        out.append(v[pages].transpose(0, 2, 1, 3, 4).reshape(cache.B, cache.Hkv, T, cache.d))
    return out[0], out[1], mapped


def _attend(cache, q, lens, counts=None, scale=None, out_dtype=None, stream=None):
    scale = cache.d ** -0.5 if scale is None else scale
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(cache, q.shape[2], q.shape[1]))
    ws.fill_(float("nan"))  # the call may not read what it has not written
    tq.tq_decode_attention_mx(q, cache, _i32(lens), scale, out, ws, None if counts is None else _i32(counts), stream)
    return out


def _check(cache, q, lens, counts=None, scale=None, out_dtype=None):
    out = _attend(cache, q, lens, counts, scale, out_dtype)
    k, v, mapped = _dense(cache)
    cnt = [q.shape[1]] * cache.B if counts is None else counts
    att = M.Attention(_np(q), k, v, mapped, lens, cnt, cache.d ** -0.5 if scale is None else scale)
    err = np.abs(_np(out) - att.o)
    tol = _bound(att, cache.d, max(max(lens), 1), out.dtype)
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-30)):.3f} of the bound"
    return out


@pytest.mark.parametrize("d,Hkv,G,Lq,page,lens,dtype,out_dtype", [
    (128, 2, 4, 1, 64, [1, 500, 17, 640, 333], "bf16", "bf16"),
    (128, 1, 8, 1, 16, [15, 16, 32, 1, 129], "f16", "f32"),
    (128, 3, 1, 1, 32, [40], "bf16", "f32"),
    (64, 12, 1, 1, 16, [300, 1, 77], "f16", "f16"),
    (64, 2, 5, 3, 128, [250, 3, 129, 64], "bf16", "f32"),      # 15 rows: two column tiles
    (256, 2, 2, 1, 64, [200, 65, 1], "bf16", "bf16"),
    (256, 1, 3, 4, 16, [90, 4, 100], "f16", "f32"),            # 12 rows in two blocks
    (128, 2, 4, 5, 16, [100, 5, 47, 16], "bf16", "f32"),       # 20 rows: three blocks
    (128, 1, 8, 16, 32, [64, 16, 200], "f16", "f32"),          # 128 rows: eight blocks of 16
    (64, 1, 7, 2, 16, [31, 33], "f16", "bf16"),
    (64, 2, 6, 4, 32, [120, 33, 4, 64], "bf16", "f32"),        # 24 rows: three blocks
    (128, 1, 11, 2, 16, [15, 16, 17, 31, 32, 33, 48, 65], "bf16", "f16"),  # 22 rows; ends within a step of 32
    (64, 3, 2, 1, 64, [15, 16, 17, 31, 32, 33, 48, 63, 65, 96], "f16", "f32"),
    (256, 2, 8, 1, 128, [1000, 31, 130], "f16", "f32"),
    (128, 8, 4, 1, 64, [3000], "bf16", "f32"),                 # few units, many CTAs each
    (64, 1, 1, 1, 16, [20000], "bf16", "f32"),                 # one unit over all CTAs
    (128, 4, 4, 1, 16, [7] * 100, "bf16", "f32"),              # many units, one tile each
])
def test_attention_matches_oracle(d, Hkv, G, Lq, page, lens, dtype, out_dtype):
    B = len(lens)
    cache = _setup(B, Hkv, d, page, lens, seed=d + Lq, g=(0.5, 2.0))
    q = _randn((B, Lq, Hkv * G, d), DT[dtype], 5, loud=False).cuda()
    _check(cache, q, lens, out_dtype=DT[out_dtype])


@pytest.mark.parametrize("Lq,G", [(1, 4), (4, 4), (7, 2), (16, 1)])
def test_attention_of_ragged_rows_and_empty_ones(Lq, G):
    # lengths of zero, counts of zero, fewer positions than queries, and counts outside 0..Lq
    lens, counts = [0, 50, 2, 40, 33, 1, 64], [Lq, 0, Lq, max(Lq - 2, 1), 99, 1, -3]
    cache = _setup(len(lens), 2, 128, 16, lens)
    q = _randn((len(lens), Lq, 2 * G, 128), torch.bfloat16, 6).cuda()
    out = _check(cache, q, lens, counts, out_dtype=torch.float32)
    assert (out[0] == 0).all() and (out[1] == 0).all() and (out[6] == 0).all()
    if Lq > 2:
        assert (out[2, :Lq - 2] == 0).all() and (out[2, Lq - 1] != 0).any()


def test_attention_over_unmapped_pages_and_past_the_table():
    lens = [70, 64, 48, 200, 30]
    cache = _setup(5, 2, 128, 16, 4, seed=9)  # 64 positions each
    bt = cache.block_table
    bt[0, 1], bt[1, 0], bt[1, 3], bt[4, 0], bt[4, 1] = -1, cache.num_pages, -7, -1, -1
    q = _randn((5, 3, 8, 128), torch.bfloat16, 7).cuda()
    out = _check(cache, q, lens, out_dtype=torch.float32)
    assert (out[4] == 0).all()  # every position it could see is unmapped


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_scales_and_sharp_rows(scale):
    cache = _setup(2, 2, 128, 32, [200, 77], seed=11, k_gain=1.0)
    q = (_randn((2, 1, 8, 128), torch.float32, 8) * 4).to(torch.bfloat16).cuda()
    _check(cache, q, [200, 77], scale=scale, out_dtype=torch.float32)


@pytest.mark.parametrize("mag", [1e-30, 1e30, 2.0 ** -133])
def test_attention_of_extreme_queries(mag):
    # bf16 queries far outside fp16's range: the scale brings the scores back
    cache = _setup(2, 1, 128, 32, [200, 77], seed=12)
    q = (_randn((2, 1, 4, 128), torch.float32, 9, loud=False) * mag).to(torch.bfloat16).cuda()
    _check(cache, q, [200, 77], scale=min(0.1 / mag, 3e38), out_dtype=torch.float32)


def test_rising_scores_move_the_reference():
    # every tile's scores pass the ones before by far more than a weight can hold
    cache = _setup(1, 1, 64, 16, 8, seed=13)
    K = torch.zeros(1, 1, 128, 64)
    K[0, 0, :, 0] = torch.arange(128) * 6.0
    V = _randn((1, 1, 128, 64), torch.float32, 14, loud=False)
    tq.tq_quantize_kv_mx(K.cuda(), V.cuda(), cache, _i32([128]))
    q = torch.zeros(1, 1, 2, 64, dtype=torch.float16)
    q[0, 0, 0, 0], q[0, 0, 1, 0] = 1.0, -1.0
    _check(cache, q.cuda(), [128], scale=4.0, out_dtype=torch.float32)


# ------------------------------------------------------------------ NaN and infinities
def _poison(cache, b, pos, side, element):
    """Make the block of one row that holds `element` NaN, in every head."""
    page = int(cache.block_table[b, pos // cache.page_size])
    cache[f"{side}_scales"][page, :, pos % cache.page_size, element // 16] = 0x7F


@pytest.mark.parametrize("d,G", [(64, 4), (128, 4), (256, 2)])
def test_what_a_query_does_not_see_cannot_reach_it(d, G):
    lens, Lq = [37, 20, 64], 4
    cache = _setup(3, 2, d, 16, 4, seed=20)
    q = _randn((3, Lq, 2 * G, d), torch.bfloat16, 21, loud=False).cuda()
    clean = _attend(cache, q, lens, out_dtype=torch.float32)
    for b, L in enumerate(lens):  # rows behind the last sequence, to the end of the table
        for pos in range(L, 64):
            for e in range(0, d, 16):
                _poison(cache, b, pos, "k", e)
                _poison(cache, b, pos, "v", e)
    assert torch.equal(clean, _attend(cache, q, lens, out_dtype=torch.float32))
    # the newest token is NaN: only the last query sees it, and only in its own values
    for b, L in enumerate(lens):
        _poison(cache, b, L - 1, "v", 16)
        _poison(cache, b, L - 2, "v", 0)
    got = _check_nan(cache, q, lens)
    assert not torch.isnan(got[:, : Lq - 2]).any()
    assert torch.isnan(got[:, Lq - 2, :, :16]).all() and not torch.isnan(got[:, Lq - 2, :, 16:]).any()
    assert torch.isnan(got[:, Lq - 1, :, :32]).all() and not torch.isnan(got[:, Lq - 1, :, 32:]).any()
    _poison(cache, 1, 17, "k", 0)  # a NaN key: every query that sees it loses its whole row
    got = _check_nan(cache, q, lens)
    assert torch.isnan(got[1, 1:]).all() and not torch.isnan(got[1, 0]).any()


def _check_nan(cache, q, lens):
    out = _attend(cache, q, lens, out_dtype=torch.float32)
    k, v, mapped = _dense(cache)
    att = M.Attention(_np(q), k, v, mapped, lens, [q.shape[1]] * cache.B, cache.d ** -0.5)
    got = _np(out)
    assert np.array_equal(np.isnan(got), np.isnan(att.o))
    ok = ~np.isnan(att.o) & np.isfinite(att.m)
    assert (np.abs(got - att.o)[ok] <= _bound(att, cache.d, max(lens), out.dtype)[ok]).all()
    return out


def test_unmapped_pages_of_nan_do_not_reach_a_row():
    cache = _setup(1, 1, 128, 16, 4, seed=23)
    for t in ("k_scales", "v_scales"):
        cache[t][0] = 0x7F  # what an unmapped entry might be read as
    bt = cache.block_table
    bt[0] = torch.where(bt[0] == 0, cache.num_pages - 1, bt[0])
    q = _randn((1, 2, 4, 128), torch.float16, 24).cuda()
    bt[0, 1] = -1
    _check(cache, q, [60], out_dtype=torch.float32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_query_row_stays_alone(bad):
    cache = _setup(2, 2, 128, 32, [90, 40], seed=25)
    q = _randn((2, 2, 8, 128), torch.bfloat16, 26).cuda()
    q[0, 1, 3, 5] = bad
    got = _check_nan(cache, q, [90, 40])
    assert torch.isnan(got[0, 1, 3]).all() and int(torch.isnan(got).any(-1).sum()) == 1


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,out_dtype", [(64, "f32"), (128, "bf16"), (256, "f16")])
def test_scores_that_are_all_minus_infinity_give_nan(d, out_dtype, dtype):
    # keys of one sign in a channel, infinite queries there: every visible score is the same infinity, and
    # the softmax of such a row is NaN for either sign. 1 and 20 positions: one warp; 100: one CTA; 3000:
    # several CTAs, joined by the combine kernel.
    lens, Lq, G = [1, 20, 100, 3000], 3, 4
    cache = _cache(4, 1, d, 16, 188, seed=27)
    K = _randn((4, 1, 3008, d), torch.float32, 28, loud=False)
    K[..., 0] = 4.0  # no code of it is 0
    tq.tq_quantize_kv_mx(K.cuda(), K.cuda(), cache, _i32([3008] * 4))
    q = _randn((4, Lq, G, d), DT[dtype], 29, loud=False).cuda()
    q[:, :, 1, 0], q[:, :, 2, 0] = float("-inf"), float("inf")
    bt = cache.block_table
    clean = _attend(cache, q, lens, out_dtype=DT[out_dtype])
    got = _np(clean)
    for b, L in enumerate(lens):
        for i in range(Lq):
            sees = L - Lq + i >= 0
            assert np.isnan(got[b, i, 1:3]).all() if sees else (got[b, i] == 0).all()
            assert np.isfinite(got[b, i, [0, 3]]).all()
    # unmapped pages first: the queries that see no mapped position stay zeros
    bt[1, 0] = bt[2, 0] = -1
    bt[3, :150] = cache.num_pages
    out = _np(_attend(cache, q, [1, 18, 18, 2402], out_dtype=DT[out_dtype]))
    for b in (1, 2, 3):
        assert (out[b, 0] == 0).all() and np.isnan(out[b, 1:, 1:3]).all() and np.isfinite(out[b, 1:][:, [0, 3]]).all()
    bt[3] = -1  # and nothing mapped at all
    assert (_np(_attend(cache, q, [1, 18, 18, 2402], out_dtype=DT[out_dtype]))[3] == 0).all()


@pytest.mark.parametrize("split", [10, 100, 1500])
def test_scores_of_minus_infinity_have_no_weight_beside_finite_ones(split):
    # scale * score passes fp32 below zero for the first positions, whole tiles and stretches of warps
    # among them, and is 0 for the others
    T = 2 * split
    cache = _cache(1, 1, 128, 16, -(-T // 16), seed=31)
    K = torch.zeros(1, 1, T, 128)
    K[0, 0, :split, 0] = 6.0
    V = _randn((1, 1, T, 128), torch.float32, 32, loud=False)
    tq.tq_quantize_kv_mx(K.cuda(), V.cuda(), cache, _i32([T]))
    q = torch.zeros(1, 1, 2, 128, dtype=torch.float16, device="cuda")
    q[0, 0, 0, 0] = -1.0
    got = _np(_attend(cache, q, [T], scale=1e38, out_dtype=torch.float32))
    v = _dense(cache)[1][0, 0, :T]
    for row, see in ((0, v[split:]), (1, v)):
        # equal weights: exact in fp16, so what rounds is T sums and the merges (2^-23 each) and the division
        tol = np.abs(see).mean(0) * (T + 64) * 2.0 ** -23 * 2 + np.abs(see.mean(0)) * 2.0 ** -21
        assert (np.abs(got[0, 0, row] - see.mean(0)) <= tol).all()


# ------------------------------------------------------------------ how it is called
def test_attention_repeats_bit_for_bit_and_shares_a_workspace_in_turn():
    cache = _setup(4, 4, 128, 32, [3000, 1, 700, 64], seed=30)
    q = _randn((4, 1, 16, 128), torch.bfloat16, 31).cuda()
    big = _attend(cache, q, [3000, 1, 700, 64])
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(cache, 16))
    outs = [torch.empty_like(q) for _ in range(6)]
    for i, o in enumerate(outs):  # calls of other lengths in between use the same workspace
        tq.tq_decode_attention_mx(q, cache, _i32([3000, 1, 700, 64] if i % 2 == 0 else [5, 0, 2999, 17]), 128 ** -0.5, o, ws)
    assert all(torch.equal(o, big) for o in outs[::2]) and torch.equal(outs[1], outs[5])


def test_captured_step_follows_lengths_and_tables():
    B, Hkv, d, page = 3, 2, 128, 16
    cache = _cache(B, Hkv, d, page, 6, seed=32)
    cache.block_table.copy_(_table(B, 6, cache.num_pages, 33))
    other = _cache(B, Hkv, d, page, 6, seed=34)
    other.block_table.copy_(cache.block_table)
    lens, counts = _i32([0] * B), _i32([0] * B)
    k, v = (torch.zeros(B, Hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, 16, 4, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(cache, 4, 16))

    def step():
        tq.tq_quantize_kv_mx(k, v, cache, lens, counts)
        tq.tq_decode_attention_mx(q, cache, lens, d ** -0.5, out, ws, counts)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    now = [0] * B
    for i in range(7):
        n = [(3 * i + b) % 17 for b in range(B)]
        now = [a + b for a, b in zip(now, n)]
        now = [min(a, 96) for a in now]
        if i == 4:  # the pages move: the table is read anew
            for key in cache.tensors:
                cache[key].copy_(cache[key].roll(1, 0))
            cache.block_table.copy_((cache.block_table + 1) % cache.num_pages)
            other.block_table.copy_(cache.block_table)
            for key in other.tensors:
                other[key].copy_(other[key].roll(1, 0))
        k.copy_(_randn(k.shape, k.dtype, 40 + i))
        v.copy_(_randn(v.shape, v.dtype, 50 + i))
        q.copy_(_randn(q.shape, q.dtype, 60 + i))
        lens.copy_(_i32(now))
        counts.copy_(_i32(n))
        g.replay()
        tq.tq_quantize_kv_mx(k, v, other, lens, counts)
        want = _attend(other, q, now, n)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for key in cache.tensors:
            assert torch.equal(cache[key], other[key])


def test_calls_on_two_streams_with_their_own_workspaces():
    caches = [_setup(4, 4, 128, 32, [2000, 3, 900, 64], seed=70 + i) for i in range(2)]
    qs = [_randn((4, 2, 16, 128), torch.bfloat16, 80 + i).cuda() for i in range(2)]
    want = [_attend(c, q, [2000, 3, 900, 64]) for c, q in zip(caches, qs)]
    lens = _i32([2000, 3, 900, 64])
    wss = [tq.workspace(tq.tq_decode_mx_workspace_bytes(c, 16, 2)) for c in caches]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, q, o, w, s in zip(caches, qs, outs, wss, streams):
            tq.tq_decode_attention_mx(q, c, lens, 128 ** -0.5, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_records_past_the_32_bit_byte_offset():
    # 2^27 records of 64 code bytes: offsets pass 2^33
    page, Hkv = 64, 8
    num_pages = (1 << 27) // (page * Hkv)
    bt = torch.tensor([[num_pages - 1, 3], [num_pages // 2 + 1, num_pages - 2]], dtype=torch.int32, device="cuda")
    cache = tq.TQMXCache(2, Hkv, 128, page, num_pages, 2, bt)
    K, V = (_randn((2, Hkv, 128, 128), torch.bfloat16, 90 + i, loud=False) for i in range(2))
    tq.tq_quantize_kv_mx(K.cuda(), V.cuda(), cache, _i32([128, 128]))
    codes, s = M.quantise(_np(K[0, Hkv - 1, 63]), 1.0)
    np.testing.assert_array_equal(cache["k_scales"][num_pages - 1, Hkv - 1, 63].cpu().numpy(), s)
    small = _cache(2, Hkv, 128, page, 2, seed=91)
    tq.tq_quantize_kv_mx(K.cuda(), V.cuda(), small, _i32([128, 128]))
    q = _randn((2, 1, 8, 128), torch.bfloat16, 92).cuda()
    assert torch.equal(_attend(cache, q, [128, 101]), _attend(small, q, [128, 101]))


def test_a_large_batch_of_short_and_empty_sequences():
    lens = [(7 * b) % 40 for b in range(700)]
    cache = _setup(700, 1, 64, 16, 3, seed=93)
    q = _randn((700, 1, 2, 64), torch.float16, 94).cuda()
    _check(cache, q, lens, out_dtype=torch.float32)


def test_bindings_refuse_wrong_tensors():
    cache = _setup(2, 2, 128, 16, 2)
    q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(cache, 4))
    lens = _i32([3, 3])
    k = torch.zeros(2, 2, 1, 128, dtype=torch.bfloat16, device="cuda")

    def refuse(f):
        with pytest.raises(tq.TQError):
            f()
    refuse(lambda: tq.tq_decode_attention_mx(q[:1], cache, lens, 0.1, q, ws))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens.long(), 0.1, q, ws))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens[:1], 0.1, q, ws))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens.cpu(), 0.1, q, ws))
    refuse(lambda: tq.tq_decode_attention_mx(q.float(), cache, lens, 0.1, q, ws))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens, 0.1, q[:, :, :2], ws))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens, 0.1, q, ws[:8]))
    refuse(lambda: tq.tq_decode_attention_mx(q, cache, lens, 0.1, q, ws, counts=lens[:1]))
    refuse(lambda: tq.tq_decode_mx_workspace_bytes(cache, 3))
    refuse(lambda: tq.tq_quantize_kv_mx(k[:, :1], None, cache, lens))
    refuse(lambda: tq.tq_quantize_kv_mx(k, k.half(), cache, lens))
    refuse(lambda: tq.tq_quantize_kv_mx(k, k.expand(2, 2, 2, 128), cache, lens))
    refuse(lambda: tq.tq_quantize_kv_mx(k.int(), None, cache, lens))
    wide = torch.zeros(2, 2, 1, 256, dtype=torch.bfloat16, device="cuda")
    refuse(lambda: tq.tq_quantize_kv_mx(wide[..., ::2], None, cache, lens))    # elements not adjacent
    refuse(lambda: tq.tq_quantize_kv_mx(wide[..., 1:129], None, cache, lens))  # not 16-byte aligned
    refuse(lambda: tq.tq_dequantize_mx(cache, lens, wide[..., :128], None))    # output not contiguous
    refuse(lambda: tq.TQMXCache(2, 2, 96, 16, 4, 2, cache.block_table))
    refuse(lambda: tq.TQMXCache(2, 2, 128, 16, 4, 2, cache.block_table, k_scale=0.0))
