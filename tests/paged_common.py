"""Shared pieces of the paged-cache tests: a cache and its oracle stepped
together, and the bounds their results are compared with."""

import numpy as np
import torch

from gpu_common import f64
from oracle import paged as opaged
from video_diffusion_transformer_self_b200 import inputs, paged, wan


def make(streams, grid, n_pages, page_size, max_pages, heads, kv_heads,
         token_cap, max_new=None, device="cuda"):
    """(PagedCache, oracle Cache) of the same sizes, both empty."""
    max_new = token_cap if max_new is None else max_new
    c = paged.PagedCache(
        torch.tensor(streams, dtype=torch.int32, device=device),
        wan.grid(*grid), n_pages=n_pages, page_size=page_size,
        max_pages=max_pages, heads=heads, kv_heads=kv_heads,
        token_cap=token_cap, max_new=max_new)
    return c, opaged.Cache(streams, grid, n_pages, page_size, max_pages,
                           token_cap, max_new)


def shuffle_ring(c, oc, seed):
    """The free pages in a random order, from a random place of the ring."""
    rng = np.random.default_rng(seed)
    oc.ring = [int(p) for p in rng.permutation(oc.n_pages)]
    oc.head = int(rng.integers(oc.n_pages))
    c.free_ring.copy_(torch.tensor(oc.ring, dtype=torch.int32))
    c.ring_state.copy_(torch.tensor([oc.head, oc.count], dtype=torch.int32))


def step(c, oc, new_lens):
    """Plans the step on both; returns the oracle's results."""
    c.plan(torch.tensor(new_lens, dtype=torch.int32, device=c.device))
    return oc.plan(new_lens)


def assert_plan(c, oc, want, what=""):
    q_start, q_lens, status, tokens = want
    for name, got, ref in (
            ("kv_lens", c.kv_lens, oc.kv), ("first_pages", c.first_pages,
                                            oc.first),
            ("block_table", c.block_table, oc.table),
            ("ring_state", c.ring_state, [oc.head, oc.count]),
            ("free_ring", c.free_ring, oc.ring),
            ("q_start", c.q_start, q_start), ("q_lens", c.q_lens, q_lens),
            ("status", c.status, status), ("tokens", c.tokens, tokens)):
        got, ref = got.cpu().numpy(), np.asarray(ref)
        assert np.array_equal(got, ref), (what, name, got, ref)


def assert_write(got, want, extra, what):
    """bf16 results of a short fp32 chain: half a step (2^-8 of the value)
    and the chain's own roundings.  A value is x f w c -+ x' f w' s: 5
    roundings of either product, the sum's, and f's relative error (the sum
    of squares over n terms in a tree of depth < 32 + 20 additions, rsqrt
    within 2 units): under 64 x 2^-24 of |x f w| + |x' f w'|, `extra`."""
    err = np.abs(got - want)
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * extra + 1e-30
    assert np.all(np.isfinite(got)), what
    assert np.all(err <= bound), (what, float(np.max(err / bound)))


def assert_attn(got, want, mag, what, score_sum):
    """o = sum w_j v_j with A = sum w_j |v_j| (`mag`).  Roundings: the
    weights to bf16, 2^-8 each, in the numerator only: 2^-8 A; the
    exponential's approximation 1.3e-4 (numerator and row sum: twice); the
    scores in fp32: 128 products and additions of |q_c k_c| and the scaling,
    at most 130 x 2^-24 x score_sum in the exponent (score_sum >= scale
    sum_c |q_c k_c|; numerator and row sum: twice); O and the row sum in
    fp32 over the keys, at most 2^-24 a key: 2^-9 / 8 for 4,096 keys a
    running sum; the result to bf16: 2^-8 |o|."""
    rel = 2.0 ** -8 + 2.6e-4 + 260 * 2.0 ** -24 * score_sum + 2.0 ** -12
    bound = rel * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    assert np.all(err <= bound), (what, float(np.max(err / bound)))


def rows_bf16(rows, heads, seed, scale=1.0):
    return inputs.randn_bf16((rows, heads, 128), seed, scale)


def expect_attn(c, oc, q, kp, vp, want, scale):
    """Oracle output of every planned row: (rows, o, mag) lists."""
    q_start, q_lens, _, _ = want
    kp64, vp64, q64 = f64(kp), f64(vp), f64(q)
    out = []
    for r, n in enumerate(q_lens):
        if n:
            rows = slice(q_start[r], q_start[r] + n)
            o, mag = opaged.attention(
                q64[rows], kp64, vp64, oc.table[r], oc.kv[r],
                oc.streams[r][2], oc.streams[r][3], scale, oc.ps)
            out.append((r, rows, o, mag))
    return out
