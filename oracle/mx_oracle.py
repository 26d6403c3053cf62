"""Plain CPU oracle of the microscaled 4-bit paged cache and of the page pool (test infrastructure
only): formats bit by bit, attention in float64, page bookkeeping as Python loops."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    """The 128 non-negative E4M3 numbers by their byte; 0x7F is NaN."""
    v = np.empty(128)
    for byte in range(128):
        e, m = byte >> 3, byte & 7
        v[byte] = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    v[0x7F] = np.nan
    return v


_E4M3 = e4m3_values()


def _nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest grid value (ascending from 0) for x >= 0, ties to the even index,
    saturating at the last."""
    hi = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2  # exact: the grids have few significant bits
    up = (x > mid) | ((x == mid) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x: np.ndarray, g: float, wide: type = np.float64):
    """x [..., d] -> (codes [..., d] of 0..15, scale bytes [..., d/16]). ``wide`` is the type of the
    two divisions: float64 for the definition, float32 for the library's arithmetic where g is no
    power of two."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    finite = np.isfinite(blocks).all(-1)
    safe = np.where(finite[..., None], blocks, 0.0).astype(wide)
    g = wide(g)
    top = np.abs(safe).max(-1)
    s = _nearest_even((top / (wide(6.0) * g)).astype(np.float64), _E4M3[:127])
    step = (_E4M3[s].astype(wide) * g)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(step > 0, safe / step, 0.0)
    mag = _nearest_even(np.abs(u).astype(np.float64), E2M1)
    codes = np.where((u < 0), mag + 8, mag)
    return codes.reshape(x.shape).astype(np.uint8), np.where(finite, s, 0x7F).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def values(packed: np.ndarray, scales: np.ndarray, g: float) -> np.ndarray:
    codes = unpack(packed)
    mag = np.where(codes >= 8, -E2M1[codes & 7], E2M1[codes & 7]).reshape(*scales.shape, 16)
    s = np.where(scales >= 0x80, -_E4M3[scales & 0x7F], _E4M3[scales & 0x7F])
    return (mag * (s * np.float64(np.float32(g)))[..., None]).reshape(codes.shape)


class Attention:
    """o [B][Lq][Hq][d] in float64, and what bounds its rounding: a = sum_j p_j |v_j|, m = the
    largest sum_i |scale q_i k_ji| of a row, v = the largest |v_j|."""

    def __init__(self, q, k_vals, v_vals, mapped, lens, counts, scale):
        # q [B, Lq, Hq, d]; k_vals, v_vals [B, Hkv, T, d]; mapped [B, T]
        B, Lq, Hq, d = q.shape
        Hkv = k_vals.shape[1]
        self.o = np.zeros(q.shape)
        self.a = np.zeros(q.shape)
        self.v = np.zeros(q.shape)
        self.m = np.zeros((B, Lq, Hq, 1))
        for b in range(B):
            n = int(np.clip(counts[b], 0, Lq))
            for i in range(n):
                upto = min(max(int(lens[b]) - n + i + 1, 0), k_vals.shape[2])
                see = np.nonzero(mapped[b, :upto])[0]
                if len(see) == 0:
                    continue
                for hq in range(Hq):
                    h = hq // (Hq // Hkv)
                    k, v = k_vals[b, h, see], v_vals[b, h, see]
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (k @ q[b, i, hq])
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        self.o[b, i, hq] = p @ v
                        self.a[b, i, hq] = p @ np.abs(v)
                        self.v[b, i, hq] = np.abs(v).max(0)
                        self.m[b, i, hq] = (np.abs(scale) * (np.abs(k) @ np.abs(q[b, i, hq]))).max()


class Pages:
    """The page pool's bookkeeping, one entry at a time. ``pools``: arrays [num_pages, ...]."""

    def __init__(self, B, max_pages, num_pages, page_size, pools=()):
        self.ps, self.max_pages = page_size, max_pages
        self.refs = np.zeros(num_pages, np.int32)
        self.table = np.full((B, max_pages), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.pools = list(pools)

    def _n(self, length):
        return -(-int(length) // self.ps)

    def extend(self, need):
        for b, n in enumerate(self.lens):  # pages behind a length that the caller lowered go back first
            for j in range(self._n(max(int(n), 0)), self.max_pages):
                if 0 <= self.table[b, j] < len(self.refs):
                    self.refs[self.table[b, j]] -= 1
                    self.table[b, j] = -1
        after = [int(n) + max(int(x), 0) for n, x in zip(self.lens, need)]
        if any(a > self.max_pages * self.ps for a in after):
            return 2
        free = iter(np.nonzero(self.refs == 0)[0])
        take = [(b, j) for b, a in enumerate(after) for j in range(self._n(self.lens[b]), self._n(a))]
        if len(take) > int((self.refs == 0).sum()):
            return 1
        for b, j in take:
            p = next(free)
            self.table[b, j], self.refs[p] = p, 1
        self.lens[:] = after
        return 0

    def fork(self, parent_of):
        B = len(self.lens)
        kids = [(b, int(p)) for b, p in enumerate(parent_of) if 0 <= p < B and p != b]
        partial = [(b, p) for b, p in kids if self.lens[p] % self.ps]
        free = np.nonzero(self.refs == 0)[0]
        if len(partial) > len(free):
            return 1
        fresh = {b: f for (b, _), f in zip(partial, free)}
        table, lens = self.table.copy(), self.lens.copy()
        for b, _ in kids:
            for e in table[b]:
                if 0 <= e < len(self.refs):
                    self.refs[e] -= 1
        for b, p in kids:
            n = self._n(lens[p])
            self.table[b] = -1
            self.table[b, :n] = table[p, :n]
            self.lens[b] = lens[p]
            if b in fresh:
                src = self.table[b, n - 1]
                self.table[b, n - 1] = fresh[b]
                for pool in self.pools:
                    if 0 <= src < len(self.refs):
                        pool[fresh[b]] = pool[src]
            for e in self.table[b]:
                if 0 <= e < len(self.refs):
                    self.refs[e] += 1
        return 0

    def free(self, leaving):
        for b, gone in enumerate(leaving):
            if gone:
                for e in self.table[b]:
                    if 0 <= e < len(self.refs):
                        self.refs[e] -= 1
                self.table[b], self.lens[b] = -1, 0

    def compact(self):
        n = int((self.refs != 0).sum())
        src = [p for p in range(len(self.refs) - 1, n - 1, -1) if self.refs[p] != 0]
        dst = [p for p in range(n) if self.refs[p] == 0]
        new = {}
        for s, t in zip(src, dst):
            new[s] = t
            self.refs[t], self.refs[s] = self.refs[s], 0
            for pool in self.pools:
                pool[t] = pool[s]
        for e in np.nditer(self.table, op_flags=["readwrite"]):
            e[...] = new.get(int(e), int(e))
        return n
