"""Paged K / V cache: the plan of a step, the write of its tokens and the
attention over the pages, one stream after another in plain Python / fp64.

Long-video survey, section "Route 3 · Self Forcing": chunk after chunk
against a KV cache, which may be capped (the H200 table caps it at 42 latent
frames).  A query at position a of a stream sees the keys
max(0, e - window) <= j < min(kv, e), e = (a // chunk + 1) * chunk.  The
paging is this library's own (the pages have no counterpart): position a lies
in row a % page_size of page table[a // page_size].
"""

import numpy as np

from . import rope as _rope

OK, EINVAL, ENOSPACE = 0, -1, -6


def visible(a, kv, chunk, window):
    """(first key, one past the last) of the query at position a."""
    e = (a // chunk + 1) * chunk
    lo = max(0, e - window) if window else 0
    return lo, max(lo, min(kv, e))


class Cache:
    """State of a paged cache with Python integers."""

    def __init__(self, streams, grid, n_pages, page_size, max_pages,
                 token_cap, max_new):
        self.streams = [tuple(s) for s in streams]
        self.grid, self.n_pages, self.ps = tuple(grid), n_pages, page_size
        self.max_pages, self.cap, self.max_new = max_pages, token_cap, max_new
        R = len(streams)
        self.kv, self.first = [0] * R, [0] * R
        self.table = [[-1] * max_pages for _ in range(R)]
        self.ring = list(range(n_pages))
        self.head, self.count = 0, n_pages

    def _pages(self, n):
        return -(-n // self.ps)

    def _push(self, page):
        self.ring[(self.head + self.count) % self.n_pages] = page
        self.count += 1

    def plan(self, new_lens):
        """q_start, q_lens, status, tokens of the step."""
        R, ps = len(self.kv), self.ps
        F, GH, GW = self.grid
        start, at = [], 0
        for n in new_lens:
            start.append(at)
            at += max(n, 0)
        fit = []
        for r, n in enumerate(new_lens):
            H, W, chunk, window = self.streams[r]
            total = self.kv[r] + max(n, 0)
            fit.append(1 <= H <= GH and 1 <= W <= GW and chunk >= 1
                       and window >= 0 and n <= self.max_new
                       and total <= self.max_pages * ps
                       and total <= F * H * W
                       and start[r] + max(n, 0) <= self.cap)
        for r, n in enumerate(new_lens):
            upto = self.first[r]
            if n < 0:
                upto = self._pages(self.kv[r])
            elif n > 0 and fit[r]:
                lo, _ = visible(self.kv[r], 1 << 40, *self.streams[r][2:])
                upto = max(upto, min(lo, self.kv[r]) // ps)
            for p in range(self.first[r], upto):
                self._push(self.table[r][p])
                self.table[r][p] = -1
            self.first[r] = upto
            if n < 0:
                self.kv[r] = self.first[r] = 0
        q_lens, status = [0] * R, [OK] * R
        tokens = [(0, 0, 0, -1)] * self.cap
        asked, stopped = 0, False
        have = self.count
        for r, n in enumerate(new_lens):
            if n <= 0:
                continue
            if not fit[r]:
                status[r] = EINVAL
                continue
            p0, p1 = self._pages(self.kv[r]), self._pages(self.kv[r] + n)
            asked += p1 - p0
            stopped = stopped or asked > have
            if stopped:
                status[r] = ENOSPACE
                continue
            for p in range(p0, p1):
                self.table[r][p] = self.ring[self.head]
                self.head = (self.head + 1) % self.n_pages
                self.count -= 1
            H, W = self.streams[r][:2]
            for i in range(n):
                a = self.kv[r] + i
                tokens[start[r] + i] = (
                    a // (H * W), a % (H * W) // W, a % W,
                    self.table[r][a // ps] * ps + a % ps)
            self.kv[r] += n
            q_lens[r] = n
        q_start = [min(x, self.cap) for x in start + [at]]
        return q_start, q_lens, status, tokens


def norm_rope_rows(x, w, pos, eps=1e-6, theta=10000.0):
    """RMSNorm over heads * 128 with weights, then the 3D RoPE at pos
    [rows, 3]; x [rows, heads, 128] fp64."""
    n, heads, d = x.shape
    ms = np.mean(x.reshape(n, -1) ** 2, axis=1)
    y = x / np.sqrt(ms + eps)[:, None, None] * w.reshape(1, heads, d)
    t, h, wd = _rope.band_widths(d)
    ang = []
    for axis, width in ((0, t), (1, h), (2, wd)):
        freq = theta ** (-2.0 * np.arange(width // 2) / width)
        ang.append(pos[:, axis, None] * freq)
    ang = np.concatenate(ang, axis=1)[:, None]
    z = (y[..., 0::2] + 1j * y[..., 1::2]) * np.exp(1j * ang)
    out = np.empty_like(y)
    out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def gather(pages, table_row, lo, hi, page_size):
    """Rows lo .. hi - 1 of a stream, [hi - lo, kv_heads, 128]."""
    j = np.arange(lo, hi)
    ids = np.asarray(table_row)[j // page_size]
    return pages[ids, :, j % page_size]


def attention(q, k_pages, v_pages, table_row, kv, chunk, window, scale,
              page_size):
    """(o, sum_j w_j |v_j|) of the last len(q) positions of one stream; q
    [n, heads, 128] fp64.  The second is the scale of the rounding errors."""
    n, heads, d = q.shape
    group = heads // k_pages.shape[1]
    o, mag = np.zeros_like(q), np.zeros_like(q)
    i = 0
    while i < n:                       # rows of one chunk see the same keys
        a = kv - n + i
        rows = min(n - i, (a // chunk + 1) * chunk - a)
        lo, hi = visible(a, kv, chunk, window)
        if hi > lo:
            k = gather(k_pages, table_row, lo, hi, page_size)
            v = gather(v_pages, table_row, lo, hi, page_size)
            for h in range(heads):
                s = q[i:i + rows, h] @ k[:, h // group].T * scale
                p = np.exp(s - s.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                o[i:i + rows, h] = p @ v[:, h // group]
                mag[i:i + rows, h] = p @ np.abs(v[:, h // group])
        i += rows
    return o, mag
