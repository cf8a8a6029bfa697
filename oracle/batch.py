"""Oracle of the operators around a paged batch: rotary positions and the page pool.

The rotation is the textbook one on complex numbers in float64; the pool is a plain list
simulation.  Nothing here is shared with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np


def rope_inverse(rot_dim: int, base: float, scaling: str = "plain", factor: float = 1.0, orig_len: float = 0.0,
                 slow: float = 1.0, fast: float = 32.0) -> np.ndarray:
    """Radians per position of each of the rot_dim / 2 pairs."""
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        w = np.clip((orig_len * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = w * f + (1 - w) * f / factor
    return f


def rope(x: np.ndarray, pos: np.ndarray, inv: np.ndarray, interleaved: bool, mscale: float = 1.0) -> np.ndarray:
    """x float64 [N][H][d] rotated at positions pos [N]; the last d - 2 len(inv) elements stay."""
    half = len(inv)
    first = np.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = (x[..., first] + 1j * x[..., second]) * (mscale * np.exp(1j * pos[:, None].astype(np.float64) * inv))[:, None]
    y = x.copy()
    y[..., first], y[..., second] = z.real, z.imag
    return y


class Pool:
    """Rows of pages by reference counts: what the page calls do, one request after another.

    errors: "bounds" and "pages", in the order met (a refused request changes nothing more)."""

    def __init__(self, n_seqs: int, pages_per_seq: int, n_pages: int, page_size: int):
        self.rows = [[] for _ in range(n_seqs)]
        self.refs = [0] * n_pages
        self.most, self.page = pages_per_seq, page_size
        self.errors = []

    def _drop(self, s, keep):
        for p in self.rows[s][keep:]:
            self.refs[p] -= 1
        del self.rows[s][keep:]

    def _serve(self, jobs):
        """jobs: (row, shared pages, pages to add, what to do once served), releases done."""
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        asked = 0
        for s, shared, need, done in jobs:
            asked += need
            if need and asked > len(free):
                self.errors.append("pages")
                continue
            for p in shared:
                self.refs[p] += 1
            new = free[asked - need:asked]
            for p in new:
                self.refs[p] = 1
            self.rows[s] = (shared if shared or done else self.rows[s]) + new
            if done:
                done(new)

    def resize(self, seq, length):
        jobs, seen = [], set()
        for s, n in zip(seq, length):
            want = -(-n // self.page)
            if not 0 <= s < len(self.rows) or s in seen or n < 0 or want > self.most:
                self.errors.append("bounds")
                if 0 <= s < len(self.rows):
                    seen.add(s)
                continue
            seen.add(s)
            self._drop(s, want)
            jobs.append((s, [], want - len(self.rows[s]), None))
        self._serve(jobs)

    def fork(self, parent, child, length, room):
        """Returns the copies (source page, destination page, tokens)."""
        jobs, seen, copies = [], set(), []
        named = {s for s in child if 0 <= s < len(self.rows)}
        before = [list(r) for r in self.rows]
        for f, s, n in zip(parent, child, length):
            ok = 0 <= s < len(self.rows) and s not in seen and n >= 0 and -(-(n + room) // self.page) <= self.most
            if 0 <= s < len(self.rows):
                seen.add(s)
            ok = ok and 0 <= f < len(self.rows) and f not in named and n <= len(before[f]) * self.page
            if not ok:
                self.errors.append("bounds")
                continue
            self._drop(s, 0)
            full = n // self.page

            def copied(new, f=f, n=n, full=full):
                if n % self.page:
                    copies.append((before[f][full], new[0], n % self.page))

            jobs.append((s, before[f][:full], -(-(n + room) // self.page) - full, copied))
        self._serve(jobs)
        return copies

    def compact(self):
        """Returns the moves (from page, to page)."""
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for p, h in to.items():
            self.refs[h], self.refs[p] = self.refs[p], 0
        self.refs = [max(r, 0) for r in self.refs]
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return list(to.items())
