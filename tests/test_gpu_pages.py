"""GPU tests of the page pool (extend, fork, free, compact, copy) against the oracle's loops, and of
the operators around it together, as a serving loop uses them."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as M
from tests import parity as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the GPU tier always has a device
    pytest.skip("needs a CUDA device", allow_module_level=True)

from quantized_decode_attention_kv_b200 import tq  # noqa: E402


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Both:
    """A page pool with caches on the GPU, and the oracle's pool beside it."""

    def __init__(self, B, max_pages, num_pages, page, layers=1, Hkv=1, d=64, seed=0):
        self.pool = tq.TQPagePool(B, max_pages, num_pages, page)
        self.caches = [tq.TQMXCache(B, Hkv, d, page, num_pages, max_pages, self.pool.block_table) for _ in range(layers)]
        g = torch.Generator(device="cuda").manual_seed(seed)
        for c in self.caches:
            for t in c.tensors.values():
                t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.flat = [t for c in self.caches for t in c.tensors.values()]
        self.want = M.Pages(B, max_pages, num_pages, page, [t.cpu().numpy().copy() for t in self.flat])
        self.arrays = tq.tq_page_arrays(self.caches) if layers else None
        self.ws = tq.workspace(tq.tq_pages_workspace_bytes(self.pool))
        self.ws.fill_(float("nan"))
        self.status, self.live = _i32([77]), _i32([77])

    def extend(self, need):
        tq.tq_pages_extend(self.pool, _i32(need), self.status)
        assert self.want.extend(need) == int(self.status)
        return int(self.status)

    def fork(self, parent_of):
        tq.tq_pages_fork(self.pool, self.arrays, _i32(parent_of), self.status, self.ws)
        assert self.want.fork(parent_of) == int(self.status)
        return int(self.status)

    def free(self, leaving):
        tq.tq_pages_free(self.pool, _i32(leaving))
        self.want.free(leaving)

    def compact(self):
        tq.tq_pages_compact(self.pool, self.arrays, self.live, self.ws)
        assert self.want.compact() == int(self.live)

    def same(self):
        np.testing.assert_array_equal(self.pool.lens.cpu().numpy(), self.want.lens)
        np.testing.assert_array_equal(self.pool.block_table.cpu().numpy(), self.want.table)
        np.testing.assert_array_equal(self.pool.refs.cpu().numpy(), self.want.refs)
        for a, b in zip(self.flat, self.want.pools):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("B,max_pages,num_pages,page,layers", [
    (1, 1, 1, 16, 1), (5, 7, 23, 16, 2), (40, 9, 131, 32, 1), (300, 4, 1000, 16, 0), (9, 600, 4099, 64, 1),
    (1500, 3, 5000, 16, 0), (6, 12, 64, 128, 9),  # nine layers: 36 arrays, the larger launch block
])
def test_a_random_life_matches_the_oracle(B, max_pages, num_pages, page, layers):
    rng = np.random.default_rng(B + num_pages)
    w = Both(B, max_pages, num_pages, page, layers, seed=B)
    seen = set()
    for step in range(30):
        seen.add(w.extend(np.where(rng.random(B) < 0.5, rng.integers(0, max_pages * page // 2 + 1, B), -3)))
        if step % 3 == 0:
            w.fork(np.where(rng.random(B) < 0.3, rng.integers(-2, B + 2, B), -1))
        if step % 2 == 0:
            w.free(rng.random(B) < 0.5)
        if step % 4 == 1:
            w.compact()
        if step % 7 == 0 or step == 29:
            w.same()
    assert 0 in seen or B == 1


@pytest.mark.parametrize("B,max_pages,num_pages", [(24, 3000, 40_000), (700, 900, 400_003)])
def test_large_pools_are_planned_by_several_blocks(B, max_pages, num_pages):
    # more pages than one block plans, and (400 003) more than its bit masks hold
    rng = np.random.default_rng(num_pages)
    w = Both(B, max_pages, num_pages, 16, layers=0)
    for refs in (w.pool.refs, w.want.refs):  # pages held by others all over the pool
        refs[::7] = 3
    seen = set()
    for step in range(3):
        seen.add(w.extend(rng.integers(0, max_pages * 16 // 3, B)))
        w.free(rng.random(B) < 0.3)
        w.fork(np.where(rng.random(B) < 0.2, rng.integers(0, B, B), -1))
        w.same()
    w.compact()
    w.same()
    assert 0 in seen


def test_nothing_changes_when_pages_run_out():
    w = Both(4, 8, 12, 16)
    assert w.extend([40, 20, 16, 0]) == 0
    w.same()
    assert w.extend([128, 0, 0, 0]) == 2          # would pass its row of the table
    assert w.extend([0, 100, 0, 17]) == 1         # 6 + 2 of six free pages
    assert w.extend([2 ** 31 - 1] * 4) == 2
    w.same()
    assert w.extend([0, 12, 0, 96]) == 0          # to the last page
    w.same()
    assert w.fork([-1, -1, 0, -1]) == 1           # no page left for the partial one
    w.same()
    assert w.extend([0, 0, 0, 0]) == 0 and w.extend([8, 0, 0, 0]) == 0
    w.same()


def test_huge_needs_of_many_sequences_do_not_wrap():
    w = Both(4096, 1 << 20, 64, 16, layers=0)
    # 4096 sequences x 2^20 pages: the sum of the needs is 2^32
    tq.tq_pages_extend(w.pool, torch.full((4096,), 1 << 24, dtype=torch.int32, device="cuda"), w.status)
    assert int(w.status) == 1 and int(w.pool.refs.sum()) == 0 and int(w.pool.lens.sum()) == 0


def test_fork_reads_all_parents_before_any_child():
    w = Both(6, 5, 60, 16, layers=2)
    w.extend([70, 16, 1, 33, 0, 48])
    w.fork([1, 0, 3, 2, -1, 5])      # pairs swap; a sequence is no child of itself
    w.same()
    w.fork([5, 0, 1, 2, 3, 4])       # a cycle
    w.same()
    w.fork([0, 0, 0, 0, 0, 0])       # all become the first
    w.same()
    assert (w.pool.lens == w.pool.lens[0]).all()
    w.fork([4, -1, 9, 6, -1, 4])     # an empty history of forks on top, 6 and 9 are no sequences
    w.same()


def test_pages_held_by_the_caller_stay_allocated():
    w = Both(3, 6, 30, 16)
    for refs in (w.pool.refs, w.want.refs):
        refs[4] = 2
        refs[20] = 1
    w.extend([60, 33, 0])
    assert 4 not in w.pool.block_table.cpu().numpy()
    w.same()
    w.free([1, 0, 0])
    w.compact()
    w.same()


@pytest.mark.parametrize("B,max_pages,num_pages,page", [
    (1, 4, 4, 16), (3, 6, 14, 16), (40, 9, 131, 32), (1500, 3, 5000, 16), (5, 200, 600, 64),
    (24, 900, 40_000, 16), (300, 900, 400_003, 16),  # planned by several blocks, the last beyond their bit masks
])
def test_pages_behind_a_lowered_length_go_back(B, max_pages, num_pages, page):
    """Drafts are written, some are rejected (the caller lowers lens), the next step extends: no page is
    lost, and pages that others share with the one that stepped back stay theirs."""
    rng = np.random.default_rng(B + num_pages)
    w = Both(B, max_pages, num_pages, page, layers=0)
    seen = set()
    for step in range(8 if num_pages < 10_000 else 3):
        seen.add(w.extend(np.where(rng.random(B) < 0.6, rng.integers(0, max_pages * page // 2 + 1, B), 0)))
        if step % 2 == 1:
            w.fork(np.where(rng.random(B) < 0.2, rng.integers(0, B, B), -1))
        low = np.where(rng.random(B) < 0.5, w.want.lens - rng.integers(0, 4 * page, B), w.want.lens).clip(0)
        w.want.lens[:] = low
        w.pool.lens.copy_(_i32(low))
        seen.add(w.extend(np.where(rng.random(B) < 0.5, rng.integers(0, page + 1, B), 0)))
        w.same()
        held = w.want.table[w.want.table >= 0]
        assert np.array_equal(np.bincount(held, minlength=num_pages), w.want.refs)
    assert 0 in seen
    w.free([1] * B)
    w.same()
    assert int(w.pool.refs.sum()) == 0


def test_a_page_that_goes_back_serves_the_same_call():
    w = Both(2, 4, 4, 16)
    assert w.extend([33, 16]) == 0  # all four pages
    for lens in (w.pool.lens, w.want.lens):
        lens[0] = 16
    assert w.extend([1, 1]) == 0 and int((w.pool.refs == 0).sum()) == 0
    w.same()
    for lens in (w.pool.lens, w.want.lens):
        lens[0] = 0
    assert w.extend([0, 0]) == 0 and int((w.pool.refs == 0).sum()) == 2  # no need: the pages go back all the same
    w.same()
    for lens in (w.pool.lens, w.want.lens):
        lens[1] = 3
    assert w.extend([0, 100]) == 2 and w.extend([64, 0]) == 1
    w.same()


def test_stepping_back_into_shared_pages_by_a_fork():
    # below where it forked, a sequence shares the page it would go on in: forked at the lower length into
    # an empty row it gets a copy of its own, and the row it leaves gives everything back
    w = Both(4, 6, 20, 16, layers=1)
    assert w.extend([40, 0, 0, 0]) == 0 and w.fork([-1, 0, -1, -1]) == 0
    for lens in (w.pool.lens, w.want.lens):
        lens[1] = 24  # in the second of two shared pages
    assert w.fork([-1, -1, 1, -1]) == 0
    w.free([0, 1, 0, 0])
    w.same()
    table = w.want.table
    assert table[2, 0] == table[0, 0] and table[2, 1] != table[0, 1] and w.want.refs[table[2, 1]] == 1
    assert w.extend([1, 0, 30, 0]) == 0
    w.same()


@pytest.mark.parametrize("n", [1, 5, 700])  # 700: more pairs than one launch carries
def test_copy_moves_listed_pages_only(n):
    w = Both(1, 4, 1500, 16, layers=2, d=128, Hkv=3)
    perm = np.random.default_rng(n).permutation(1500)
    dst, src = perm[:n], np.random.default_rng(n + 1).choice(perm[n:], n)  # a source may repeat
    tq.tq_pages_copy(w.arrays, src.tolist(), dst)
    for pool in w.want.pools:
        pool[dst] = pool[src]
    w.same()
    with pytest.raises(tq.TQError):
        tq.tq_pages_copy(w.arrays, [0], [0])
    with pytest.raises(tq.TQError):
        tq.tq_pages_copy(w.arrays, [0, 1], [2])
    tq.tq_pages_copy(w.arrays, [], [])
    w.same()


def test_bookkeeping_replays_from_a_graph():
    w = Both(5, 6, 40, 16)
    need, parent, leaving = _i32([0] * 5), _i32([-1] * 5), _i32([0] * 5)

    def step():
        tq.tq_pages_free(w.pool, leaving)
        tq.tq_pages_extend(w.pool, need, w.status)
        tq.tq_pages_fork(w.pool, w.arrays, parent, w.status, w.ws)
        tq.tq_pages_compact(w.pool, w.arrays, w.live, w.ws)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(3)
    for _ in range(8):
        n, p, f = rng.integers(0, 30, 5), rng.integers(-1, 5, 5), rng.integers(0, 2, 5)
        need.copy_(_i32(n))
        parent.copy_(_i32(p))
        leaving.copy_(_i32(f))
        g.replay()
        w.want.free(f)
        w.want.extend(n)
        w.want.fork(p)
        w.want.compact()
        w.same()


@pytest.mark.parametrize("B,max_pages,num_pages", [(3, 6, 9), (1500, 3, 2000), (12, 900, 20_000)])
def test_granted_counts_are_what_was_added(B, max_pages, num_pages):
    rng = np.random.default_rng(num_pages)
    w = Both(B, max_pages, num_pages, 16, layers=0)
    seen = set()
    for step in range(8):
        need = np.where(rng.random(B) < 0.7, rng.integers(-3, max_pages * 4, B), 0)
        before = w.want.lens.copy()
        asked, granted = _i32(need), _i32([99] * B)
        tq.tq_pages_extend(w.pool, asked, w.status, granted=granted)
        seen.add(w.want.extend(need))
        w.same()
        np.testing.assert_array_equal(granted.cpu().numpy(), w.want.lens - before)
        assert torch.equal(asked.cpu(), torch.tensor(need, dtype=torch.int32))
        if step % 3 == 2:
            w.free(rng.random(B) < 0.5)
    before = w.want.lens.copy()
    asked = _i32([1] * B)  # the needs' own tensor takes the counts
    tq.tq_pages_extend(w.pool, asked, w.status, granted=asked)
    w.want.extend([1] * B)
    np.testing.assert_array_equal(asked.cpu().numpy(), w.want.lens - before)
    assert 0 in seen
    granted = _i32([99] * B)  # more than a row of the table holds
    tq.tq_pages_extend(w.pool, _i32([1] * (B - 1) + [max_pages * 16 + 1]), w.status, granted=granted)
    assert int(w.status) == 2 and not granted.any()
    w.same()
    with pytest.raises(tq.TQError):
        tq.tq_pages_extend(w.pool, asked, w.status, granted=asked[:1] if B > 1 else asked.long())


def test_a_step_without_room_leaves_every_record_as_it_was():
    """A captured step (extend, write, attend) whose sequences share pages: when pages run out it writes
    nothing and attends to nothing, and goes on when there is room again."""
    B, Hkv, d, page = 3, 2, 128, 16
    pool = tq.TQPagePool(B, 6, 5, page)
    cache = tq.TQMXCache(B, Hkv, d, page, 5, 6, pool.block_table)
    arrays, ws_p = tq.tq_page_arrays(cache), tq.workspace(tq.tq_pages_workspace_bytes(pool))
    need, n, status = _i32([32, 0, 0]), _i32([0] * B), _i32([7])
    g = torch.Generator().manual_seed(8)
    x = torch.randn(B, Hkv, 32, d, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(B, 4, Hkv, d, generator=g).to(torch.bfloat16).cuda()
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(cache, Hkv, 4))
    tq.tq_pages_extend(pool, need, status, granted=n)
    tq.tq_quantize_kv_mx(x, x, cache, pool.lens, n)
    tq.tq_pages_fork(pool, arrays, _i32([-1, 0, 0]), status, ws_p)  # all three share both pages
    assert int(status) == 0 and int(pool.refs[0]) == 3
    new = torch.randn(B, Hkv, 4, d, generator=g).to(torch.bfloat16).cuda()
    out = torch.full_like(q, 5.0)

    def step():
        tq.tq_pages_extend(pool, need, status, granted=n)
        tq.tq_quantize_kv_mx(new, new, cache, pool.lens, n)
        tq.tq_decode_attention_mx(q, cache, pool.lens, d ** -0.5, out, ws, n)
    need.copy_(_i32([0, 0, 0]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    before = {k: t.clone() for k, t in cache.tensors.items()}
    for ask, want in (([4, 17, 33], 1), ([4, 4, 100], 2)):  # six pages where three are free; a row too long
        need.copy_(_i32(ask))
        out.fill_(5.0)
        graph.replay()
        assert int(status) == want and pool.lens.tolist() == [32] * 3 and n.tolist() == [0] * 3
        assert all(torch.equal(t, before[k]) for k, t in cache.tensors.items())
        assert (out == 0).all()
    need.copy_(_i32([4, 1, 3]))
    graph.replay()
    assert int(status) == 0 and n.tolist() == [4, 1, 3] and pool.lens.tolist() == [36, 33, 35]
    for side in "kv":  # the shared pages are as they were
        for p in pool.block_table[0, :2].tolist():
            assert torch.equal(cache[f"{side}_codes"][p], before[f"{side}_codes"][p])
    back = torch.empty_like(new)
    tq.tq_dequantize_mx(cache, pool.lens, back, None, n)
    assert (back[0] != 0).any(-1).all() and (back[1, :, 1:] == 0).all() and (out[2, :3] != 0).any(-1).all()


# ------------------------------------------------------------------ together
def test_a_serving_loop_of_two_layers():
    """Prompts arrive, steps are taken, one conversation is forked into samples, others leave, the pool
    is packed, drafts are verified: every step's attention equals that of the same histories kept in
    a cache of their own, position by position."""
    B, Hkv, G, d, page, layers = 6, 2, 4, 128, 16, 2
    pool = tq.TQPagePool(B, 12, 60, page)
    caches = [tq.TQMXCache(B, Hkv, d, page, 60, 12, pool.block_table) for _ in range(layers)]
    arrays, ws_p = tq.tq_page_arrays(caches), tq.workspace(tq.tq_pages_workspace_bytes(pool))
    status, live = _i32([0]), _i32([0])
    ws = tq.workspace(tq.tq_decode_mx_workspace_bytes(caches[0], Hkv * G, 16))
    gen = torch.Generator().manual_seed(5)
    history = [[torch.zeros(2, Hkv, 0, d, dtype=torch.bfloat16) for _ in range(B)] for _ in range(layers)]

    def step(counts, Lq):
        tq.tq_pages_extend(pool, _i32(counts), status)
        assert int(status) == 0
        cnt = _i32(counts)
        for layer, cache in enumerate(caches):
            kv = torch.randn(2, B, Hkv, Lq, d, generator=gen).to(torch.bfloat16)
            q = torch.randn(B, Lq, Hkv * G, d, generator=gen).to(torch.bfloat16).cuda()
            tq.tq_quantize_kv_mx(kv[0].cuda(), kv[1].cuda(), cache, pool.lens, cnt)
            for b, n in enumerate(counts):
                history[layer][b] = torch.cat([history[layer][b], kv[:, b, :, :n]], dim=2)
            if Lq > 16:
                continue
            out = torch.empty_like(q)
            tq.tq_decode_attention_mx(q, cache, pool.lens, d ** -0.5, out, ws, cnt)
            # the same histories, each written whole into a cache of its own
            lens = [h.shape[2] for h in history[layer]]
            assert lens == pool.lens.tolist()
            T = max(lens)
            own = tq.TQMXCache(B, Hkv, d, page, B * 12, 12, torch.arange(B * 12, dtype=torch.int32, device="cuda").view(B, 12))
            x = torch.zeros(2, B, Hkv, T, d, dtype=torch.bfloat16)
            for b, h in enumerate(history[layer]):
                x[:, b, :, :lens[b]] = h
            tq.tq_quantize_kv_mx(x[0].cuda(), x[1].cuda(), own, pool.lens, pool.lens)
            want = torch.empty_like(q)
            tq.tq_decode_attention_mx(q, own, pool.lens, d ** -0.5, want, ws, cnt)
            assert torch.equal(out, want)

    step([50, 3, 20, 0, 0, 0], 50)              # prompts
    step([1, 1, 1, 0, 0, 0], 1)                 # a decode step of those there
    tq.tq_pages_fork(pool, arrays, _i32([-1, -1, -1, 0, 0, 2]), status, ws_p)
    assert int(status) == 0
    for h in history:
        h[3], h[4], h[5] = h[0], h[0], h[2]
    step([1] * 6, 1)
    step([1, 5, 0, 4, 2, 5], 5)                 # drafts of different lengths
    tq.tq_pages_free(pool, _i32([1, 0, 0, 1, 0, 0]))
    for h in history:
        h[0] = h[3] = h[0][:, :, :0]
    tq.tq_pages_compact(pool, arrays, live, ws_p)
    assert int(live) == int((pool.refs != 0).sum()) and int(pool.block_table.max()) < int(live)
    step([16, 1, 1, 0, 1, 1], 16)               # a new prompt beside running ones
    step([1, 1, 1, 0, 1, 1], 1)


@pytest.mark.parametrize("prod", [False, True])
def test_pages_of_the_rotated_caches_move_too(prod):
    """Fork and compact the pages of a TQPagedCache: the records and the decode are those of a cache
    that holds the same vectors on pages of its own, at the same lengths (the decode's split goes by them)."""
    B, Hkv, page = 6, 2, 16
    d, G = (64, 2) if prod else (128, 4)
    pool = tq.TQPagePool(B, 6, 50, page)
    mode = tq.TQ_PROD if prod else tq.TQ_MSE

    def new(num_pages, table):
        return tq.TQPagedCache(B, Hkv, d, page, num_pages, 6, 2 if prod else 4, 2, table, k_mode=mode, v_mode=mode,
                               k_qjl_m=64 if prod else 0, v_qjl_m=64 if prod else 0)
    cache, own = new(50, pool.block_table), new(B * 6, torch.arange(B * 6, dtype=torch.int32, device="cuda").view(B, 6))
    arrays, ws_p = tq.tq_page_arrays(cache), tq.workspace(tq.tq_pages_workspace_bytes(pool))
    assert arrays.n == (8 if prod else 4)
    status, live = _i32([0]), _i32([0])
    g = torch.Generator().manual_seed(6)
    K, V = (torch.randn(B, Hkv, 80, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(B, Hkv * G, d, generator=g).to(torch.bfloat16).cuda()

    def check(of, lens):  # sequence b holds the first lens[b] vectors of K[of[b]], V[of[b]]
        tq.tq_quantize_kv_paged(K[of], V[of], own)
        outs = [torch.empty(q.shape, device="cuda") for _ in range(2)]
        for c, out in zip((cache, own), outs):
            ws = tq.workspace(tq.tq_decode_paged_workspace_bytes(c, q.shape[1], lens))
            tq.tq_decode_attention_paged(q, c, lens, d ** -0.5, out, ws)
        for key in ("codes", "norm", "signs", "rnorm"):
            for side in "kv":
                if cache[f"{side}_{key}"] is None:
                    continue
                for b, L in enumerate(lens):  # every record, bit by bit
                    pos = torch.arange(L, device="cuda")
                    a, w = (c[f"{side}_{key}"][c.block_table[b, pos // page].long(), :, pos % page] for c in (cache, own))
                    assert torch.equal(a, w)
        if prod:  # this decode adds its partials in the order they arrive: the same call differs in the last bits
            P.assert_attention_close(P.to_np(outs[0]), P.to_np(outs[1]))
        else:
            assert torch.equal(*outs)
    lens = [70, 33, 16, 5, 80, 80]
    tq.tq_pages_extend(pool, _i32([80] * B), status)
    tq.tq_quantize_kv_paged(K, V, cache)  # writes one length for the whole batch
    pool.lens.copy_(_i32(lens))           # the mapped pages behind are no part of what is forked
    check([0, 1, 2, 3, 4, 5], lens)
    tq.tq_pages_free(pool, _i32([0, 0, 0, 0, 1, 1]))
    tq.tq_pages_fork(pool, arrays, _i32([-1, -1, -1, -1, 0, 1]), status, ws_p)
    assert int(status) == 0 and pool.lens.tolist() == lens[:4] + lens[:2]
    check([0, 1, 2, 3, 0, 1], lens[:4] + lens[:2])
    # sequence 2 leaves, the pool is packed, 3 is forked into its place
    tq.tq_pages_free(pool, _i32([0, 0, 1, 0, 0, 0]))
    before = pool.block_table.clone()
    tq.tq_pages_compact(pool, arrays, live, ws_p)
    assert int(live) < 50 and not torch.equal(before, pool.block_table)
    tq.tq_pages_fork(pool, arrays, _i32([-1, -1, 3, -1, -1, -1]), status, ws_p)
    assert int(status) == 0
    check([0, 1, 3, 3, 0, 1], [70, 33, 5, 5, 70, 33])
