"""The paged-cache oracle against closed forms and brute force."""

import numpy as np

from oracle import attention as oattn
from oracle import block as oblock
from oracle import paged as op


def test_visible_is_the_block_causal_rule():
    for chunk in (1, 4, 5):
        for kv in (1, 7, 20):
            for a in range(kv):
                lo, hi = op.visible(a, kv, chunk, 0)
                assert lo == 0 and hi == min(kv, (a // chunk + 1) * chunk)
    # window of two chunks: the own chunk and the one before
    assert op.visible(13, 20, 4, 8) == (8, 16)
    # a window shorter than the rest of the chunk hides every written key
    assert op.visible(4, 5, 4, 2) == (6, 6)


def test_pages_are_conserved_and_never_shared():
    rng = np.random.default_rng(3)
    streams = [(2, 3, 6, int(w)) for w in rng.integers(0, 3, 9) * 6]
    c = op.Cache(streams, (200, 4, 4), 40, 16, 70, 400, 300)
    for _ in range(60):
        new = [int(x) for x in rng.integers(-2, 40, 9)]
        c.plan(new)
        held = [p for row in c.table for p in row if p >= 0]
        free = [c.ring[(c.head + i) % 40] for i in range(c.count)]
        assert sorted(held + free) == list(range(40))
        for r, row in enumerate(c.table):
            for p, page in enumerate(row):
                inside = c.first[r] <= p < -(-c.kv[r] // 16)
                assert (page >= 0) == inside


def test_attention_equals_the_contiguous_oracle():
    rng = np.random.default_rng(4)
    ps, kv, n, heads = 16, 77, 30, 2
    table = [int(x) for x in rng.permutation(9)]
    kp, vp = rng.standard_normal((2, 9, heads, ps, 128))
    q = rng.standard_normal((n, heads, 128))
    k = op.gather(kp, table, 0, kv, ps)[None]
    v = op.gather(vp, table, 0, kv, ps)[None]
    o, mag = op.attention(q, kp, vp, table, kv, 12, 0, 0.09, ps)
    want = oattn.block_causal_attention(q[None], k, v, 0.09, 12, kv - n)
    assert np.allclose(o, want[0], rtol=1e-12, atol=1e-13)
    assert np.all(mag >= np.abs(o) - 1e-12)
    # a window hides the same keys as a brute-force mask
    o, _ = op.attention(q, kp, vp, table, kv, 12, 20, 0.09, ps)
    a = np.arange(kv - n, kv)[:, None]
    j = np.arange(kv)[None]
    e = (a // 12 + 1) * 12
    s = np.einsum("ihd,jhd->hij", q, k[0]) * 0.09
    s = np.where((j < e) & (j >= e - 20), s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), v[0])
    assert np.allclose(o, want, rtol=1e-12, atol=1e-13)


def test_write_equals_the_grid_oracle():
    rng = np.random.default_rng(5)
    grid, heads = (2, 3, 4), 3
    x = rng.standard_normal((1, 24, heads, 128))
    w = rng.standard_normal(heads * 128)
    n = np.arange(24)
    pos = np.stack([n // 12, n // 4 % 3, n % 4], 1)
    want = oblock.qk_norm_rope(x, w, grid)
    got = op.norm_rope_rows(x[0], w, pos)
    assert np.allclose(got, want[0], rtol=1e-12, atol=1e-12)
