"""CPU tests of the microscaled cache and page pool: the oracle's formats and bookkeeping against
independent statements of them, and the refusals of the C entry points (all before any device
work)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mx_oracle as M

tq = pytest.importorskip("quantized_decode_attention_kv_b200.tq")

P = 4096  # a fake, 16-byte aligned "device" address: never dereferenced on these paths


# ------------------------------------------------------------------ oracle
def test_e4m3_bytes_match_torch():
    want = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(M.e4m3_values(), want)


@pytest.mark.parametrize("x,want", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0),
                                    (5.0, 4.0), (5.1, 6.0), (0.2, 0.0), (0.3, 0.5), (100.0, 6.0)])
def test_e2m1_ties_go_to_even(x, want):
    # a block whose largest element is 6 (or the probe itself, saturated) has the scale 1
    block = np.zeros(16)
    block[0], block[3], block[4] = 6.0, min(x, 6.0), -min(x, 6.0)
    codes, s = M.quantise(block, 1.0)
    v = M.values(M.pack(codes), s, 1.0)
    assert s[0] == 0x38 and v[3] == want and v[4] == -want


def test_scales_round_to_even_saturate_and_vanish():
    def scale(top, g=1.0):
        b = np.zeros(16)
        b[7] = top
        return int(M.quantise(b, g)[1][0])
    for t in np.geomspace(2.0 ** -9, 440.0, 400):
        want = int(torch.tensor(float(t)).to(torch.float8_e4m3fn).view(torch.uint8))
        assert scale(6.0 * np.float64(np.float32(t))) == want
    assert scale(6 * 1e6) == 0x7E and scale(np.inf) == 0x7F and scale(np.nan) == 0x7F
    assert scale(6 * 2.0 ** -10) == 0  # the tie between 0 and 2^-9 goes to 0
    assert scale(0.0) == 0


def test_float32_and_float64_arithmetic_agree_for_power_of_two_scales():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 64)).astype(np.float32) * np.exp(rng.standard_normal((500, 1)) * 4)
    for wide in (x.astype(np.float32), torch.from_numpy(x).bfloat16().double().numpy()):
        for g in (1.0, 0.25, 8.0):
            a, b = M.quantise(wide, g), M.quantise(wide, g, np.float32)
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_oracle_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((1, 2, 2, 8)), rng.standard_normal((1, 1, 5, 8)), rng.standard_normal((1, 1, 5, 8))
    a = M.Attention(q, k, v, np.ones((1, 5), bool), [5], [2], 0.3)
    s = torch.from_numpy(0.3 * q[0, 0] @ k[0, 0, :4].T).softmax(-1).numpy()
    np.testing.assert_allclose(a.o[0, 0], s @ v[0, 0, :4], rtol=1e-13)


def test_oracle_pages_keep_counts_and_contents():
    rng = np.random.default_rng(2)
    pool = np.arange(40) * 10
    p = M.Pages(6, 8, 40, 16, [pool])
    assert p.extend([33, 1, 0, 16, 0, 0]) == 0 and list(p.lens) == [33, 1, 0, 16, 0, 0]
    assert p.fork([-1, -1, 0, -1, 3, 7]) == 0  # 7 is no sequence
    assert p.table[2, 0] == p.table[0, 0] and p.table[2, 2] != p.table[0, 2] and p.table[4, 0] == p.table[3, 0]
    assert pool[p.table[2, 2]] == pool[p.table[0, 2]]
    assert p.extend([0, 0, 0, 0, 0, 129]) == 2 and p.extend([10 ** 6] * 6) == 2
    for _ in range(20):
        p.free(rng.integers(0, 2, 6))
        p.extend(rng.integers(0, 40, 6))
        p.fork(rng.integers(-1, 6, 6))
        n = p.compact()
        held = p.table[p.table >= 0]
        assert np.array_equal(np.bincount(held, minlength=40), p.refs) and (p.refs[n:] == 0).all() and (p.refs[:n] > 0).all()


# ------------------------------------------------------------------ refusals
def _mx(**kw):
    base = dict(B=2, Hkv=2, d=128, page_size=16, num_pages=8, max_pages=4, k_scale=1.0, v_scale=1.0, k_codes=P,
                v_codes=P, k_scales=P, v_scales=P, block_table=P)
    base.update(kw)
    return tq.tq_mx_cache(*base.values())


BAD_CACHES = [
    (dict(B=0), 1), (dict(B=65536), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(d=32), 2), (dict(d=512), 2),
    (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(max_pages=1 << 27), 1), (dict(num_pages=1 << 27), 1), (dict(k_scale=0.0), 1), (dict(v_scale=-1.0), 1),
    (dict(k_scale=float("nan")), 1), (dict(v_scale=float("inf")), 1), (dict(v_scale=2.0 ** 65), 1),
    (dict(k_codes=None), 1), (dict(v_scales=P + 8), 1), (dict(block_table=None), 1),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_mx_call_refuses_a_bad_cache(kw, status):
    c = ctypes.byref(_mx(**kw))
    assert tq.lib.tq_quantize_kv_mx(P, P, 1, 1, None, None, P, None, c, None) == status
    assert tq.lib.tq_dequantize_mx(c, 1, P, None, P, P, 1, None) == status
    assert tq.lib.tq_decode_attention_mx(P, 1, 4, 1, P, None, 0.1, c, P, 1, P, 1 << 30, None) == status
    assert tq.lib.tq_decode_mx_workspace_bytes(4, 1, c) == 0
    assert tq.lib.tq_mx_cache_arrays(c, (tq.tq_page_array * 8)()) == 0


def test_mx_row_calls_refuse_bad_arguments():
    c, lib = ctypes.byref(_mx()), tq.lib
    strides = lambda *v: ctypes.cast((ctypes.c_int64 * 3)(*v), ctypes.c_void_p)  # noqa: E731
    w = lambda **kw: lib.tq_quantize_kv_mx(*{**dict(K=P, V=P, dt=1, T=1, ks=None, vs=None, lens=P, counts=None,  # noqa: E731
                                                    c=c, s=None), **kw}.values())
    assert w(c=None) == 1 and w(K=None, V=None) == 1 and w(K=P + 2) == 1 and w(dt=3) == 1 and w(T=-1) == 1
    assert w(lens=None) == 1 and w(lens=P + 2) == 1 and w(counts=P + 1) == 1 and w(T=(1 << 30) + 1) == 1
    assert w(ks=strides(-128, 128, 128)) == 1 and w(vs=strides(128, 128, 4)) == 1 and "stride" in tq.last_error()
    assert w(T=1 << 30, c=ctypes.byref(_mx(B=65535))) == 1
    assert w(T=0) == 0  # nothing to do
    r = lambda **kw: lib.tq_dequantize_mx(*{**dict(c=c, T=1, lens=P, counts=None, K=P, V=P, dt=1, s=None),  # noqa: E731
                                            **kw}.values())
    assert r(c=None) == 1 and r(K=None, V=None) == 1 and r(V=P + 4) == 1 and r(dt=-1) == 1 and r(T=-1) == 1
    assert r(lens=None) == 1 and r(T=0) == 0


def test_mx_attention_refuses_bad_arguments():
    c, lib = ctypes.byref(_mx()), tq.lib
    a = lambda **kw: lib.tq_decode_attention_mx(*{**dict(q=P, dt=1, Hq=4, Lq=1, lens=P, counts=None, scale=0.1, c=c,  # noqa: E731
                                                         out=P, odt=1, ws=P, n=1 << 30, s=None), **kw}.values())
    assert a(q=None) == 1 and a(q=P + 8) == 1 and a(out=None) == 1 and a(lens=None) == 1 and a(counts=P + 2) == 1
    assert a(dt=0) == 2 and a(dt=9) == 1 and a(odt=5) == 1 and a(scale=float("nan")) == 1 and a(scale=float("inf")) == 1
    assert a(Hq=3) == 1 and a(Hq=0) == 1 and a(Hq=65536) == 1 and a(Lq=0) == 1 and a(Lq=17) == 1 and a(c=None) == 1
    assert lib.tq_decode_mx_workspace_bytes(3, 1, c) == 0 and lib.tq_decode_mx_workspace_bytes(4, 17, c) == 0


def _pool(**kw):
    base = dict(B=2, max_pages=4, num_pages=8, page_size=16, refs=P, block_table=P, lens=P)
    base.update(kw)
    return tq.tq_page_pool(*base.values())


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=4097), dict(max_pages=0), dict(num_pages=0), dict(page_size=8),
                                dict(page_size=24), dict(max_pages=1 << 27), dict(num_pages=(1 << 30) + 1),
                                dict(refs=None), dict(block_table=P + 4), dict(lens=None)])
def test_every_page_call_refuses_a_bad_pool(kw):
    p, lib = ctypes.byref(_pool(**kw)), tq.lib
    assert lib.tq_pages_workspace_bytes(p) == 0
    assert lib.tq_pages_extend(p, P, P, None) == 1 and lib.tq_pages_free(p, P, None) == 1
    assert lib.tq_pages_fork(p, None, 0, P, P, P, 1 << 30, None) == 1
    assert lib.tq_pages_compact(p, None, 0, P, P, 1 << 30, None) == 1


def test_page_calls_refuse_bad_arguments():
    p, lib = ctypes.byref(_pool()), tq.lib
    ws = lib.tq_pages_workspace_bytes(p)
    assert ws >= 4 * (4 + 3 * 8) and ws % 16 == 0
    one = lambda base=P, n=64: (tq.tq_page_array * 1)(tq.tq_page_array(base, n))  # noqa: E731
    assert lib.tq_pages_extend(None, P, P, None) == 1
    assert lib.tq_pages_extend(p, None, P, None) == 1 and lib.tq_pages_extend(p, P, P + 2, None) == 1
    assert lib.tq_pages_free(p, None, None) == 1
    for fn, arg in ((lib.tq_pages_fork, (P, P)), (lib.tq_pages_compact, (P,))):
        assert fn(p, one(), 1, *arg, P, ws - 1, None) == 3 and fn(p, one(), 1, *arg, None, ws, None) == 3
        assert fn(p, one(), 1, *arg, P + 4, ws, None) == 3
        for bad in (one(None), one(P + 8), one(P, 0), one(P, 24), one(P, 1 << 31)):
            assert fn(p, bad, 1, *arg, P, ws, None) == 1
        assert fn(p, one(), -1, *arg, P, ws, None) == 1 and fn(p, one(), 1025, *arg, P, ws, None) == 1
        assert fn(p, None, 1, *arg, P, ws, None) == 1
        assert fn(p, None, 0, *[None] * len(arg), P, ws, None) == 1


def test_page_copies_refuse_overlapping_or_missing_pages():
    lib = tq.lib
    one = (tq.tq_page_array * 1)(tq.tq_page_array(P, 64))

    def copy(src, dst, num_pages=8, arrays=one, n_arrays=1):
        s, d = (np.asarray(x, dtype=np.int32) for x in (src, dst))
        return lib.tq_pages_copy(arrays, n_arrays, num_pages, s.ctypes.data, d.ctypes.data, len(s), None)
    assert copy([0], [8]) == 1 and copy([-1], [2]) == 1 and copy([0], [-1]) == 1 and copy([8], [0]) == 1
    assert copy([0, 1], [2, 2]) == 1 and "destination of two" in tq.last_error()
    assert copy([0, 1], [1, 2]) == 1 and "source and a destination" in tq.last_error()
    assert copy([3], [3]) == 1
    assert copy([0], [1], num_pages=0) == 1 and copy([0], [1], n_arrays=0) == 1 and copy([0], [1], arrays=None) == 1
    assert lib.tq_pages_copy(one, 1, 8, None, None, 1, None) == 1
    assert copy([], []) == 0


def test_paged_cache_arrays_list_every_array_of_a_page():
    # keys: 2-bit TurboQuant_prod of d = 64 with 64 sketch rows; values: 3-bit codes
    c = tq.tq_paged_cache()
    c.B, c.Hkv, c.d, c.page_size, c.num_pages, c.max_pages = 1, 3, 64, 32, 4, 4
    c.kc, c.vc = tq.tq_qcfg(2, tq.TQ_PROD, 64), tq.tq_qcfg(3, tq.TQ_MSE, 0)
    for i, f in enumerate(("k_codes", "k_norm", "k_signs", "k_rnorm", "v_codes", "v_norm")):
        setattr(c, f, 0x1000 * (i + 1))
    out = (tq.tq_page_array * 8)()
    assert tq.lib.tq_paged_cache_arrays(ctypes.byref(c), out) == 6
    rows = 3 * 32
    assert [(a.base, a.page_bytes) for a in out[:6]] == [
        (0x1000, rows * 8), (0x2000, rows * 2), (0x3000, rows * 8), (0x4000, rows * 2), (0x5000, rows * 24),
        (0x6000, rows * 2)]
    c.k_norm = None
    assert tq.lib.tq_paged_cache_arrays(ctypes.byref(c), out) == 0
    assert tq.lib.tq_paged_cache_arrays(None, out) == 0


def test_bindings_refuse_host_tensors():
    with pytest.raises(tq.TQError):
        tq.TQMXCache(1, 1, 128, 16, 4, 4, torch.zeros(1, 4, dtype=torch.int32))
    cache = type("C", (), dict(B=1, Hkv=1, d=128, device=torch.device("cuda", 0), ref=ctypes.byref(_mx(B=1, Hkv=1))))()
    x = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    for call in (lambda: tq.tq_quantize_kv_mx(x, None, cache, lens), lambda: tq.tq_dequantize_mx(cache, lens, x, x),
                 lambda: tq.tq_quantize_kv_mx(None, None, cache, lens),
                 lambda: tq.tq_decode_attention_mx(x, cache, lens, 0.1, x, x)):
        with pytest.raises(tq.TQError):
            call()


@pytest.mark.parametrize("bad", [[2 ** 32], [1.5], [[1, 2]], np.array([0.0]), np.array([2 ** 33]), np.zeros((1, 1), int), ["1"]])
def test_page_lists_that_are_no_c_ints_are_refused(bad):
    with pytest.raises(tq.TQError):
        tq._host_ints(bad, "src")


def test_page_lists_of_any_integer_type():
    for x in ([3, 1], (3, 1), np.array([3, 1]), np.array([3, 9, 1, 9], np.uint8)[::2], torch.tensor([3, 1])):
        owner, address = tq._host_ints(x, "src")
        assert len(owner) == 2 and list((ctypes.c_int * 2).from_address(address)) == [3, 1]
    assert len(tq._host_ints([], "src")[0]) == 0 and len(tq._host_ints(np.array([], int), "src")[0]) == 0


def test_extend_with_granted_counts_refuses_bad_arguments():
    p, f = ctypes.byref(_pool()), tq.lib.tq_pages_extend_granted
    assert f(None, P, P, P, None) == 1 and f(ctypes.byref(_pool(B=0)), P, P, P, None) == 1
    assert f(p, None, P, P, None) == 1 and f(p, P, None, P, None) == 1 and f(p, P, P, None, None) == 1
    assert f(p, P, P + 2, P, None) == 1 and "granted" in tq.last_error()


def test_calls_of_no_rows_do_nothing():
    # the address of a tensor without elements is NULL
    c = ctypes.byref(_mx())
    assert tq.lib.tq_quantize_kv_mx(None, None, 1, 0, None, None, P, None, c, None) == 0
    assert tq.lib.tq_quantize_kv_mx(None, None, 1, 0, None, None, None, None, c, None) == 1  # lens is still checked
    assert tq.lib.tq_dequantize_mx(c, 0, P, None, None, None, 1, None) == 0
    assert tq.lib.tq_quantize_kv_mx(None, None, 1, 1, None, None, P, None, c, None) == 1
    assert tq.lib.tq_dequantize_mx(c, 1, P, None, None, None, 1, None) == 1
