"""GPU parity of the attention over paged keys and values against the fp64
oracle, on both kernels (few rows a key head, 256-row tiles)."""

import math

import numpy as np
import pytest
import torch

from gpu_common import check_guards, f64, guarded_empty_like
from paged_common import (assert_attn, expect_attn, make, rows_bf16,
                          shuffle_ring, step)
from video_diffusion_transformer_self_b200 import build, inputs, wan

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wan.lib()


def _fill(c, oc, seed):
    """Random pools; every row that no stream holds is NaN."""
    shape = (c.n_pages, c.kv_heads, c.page_size, 128)
    kp = inputs.randn_bf16(shape, seed)
    vp = inputs.randn_bf16(shape, seed + 1)
    live = torch.zeros(c.n_pages, c.page_size, dtype=torch.bool)
    for r, row in enumerate(oc.table):
        for p in range(oc.first[r], -(-oc.kv[r] // oc.ps)):
            live[row[p], :min(oc.ps, oc.kv[r] - p * oc.ps)] = True
    dead = ~live[:, None, :, None]
    nan = torch.tensor(float("nan"), dtype=torch.bfloat16)
    return torch.where(dead, nan, kp).cuda(), torch.where(dead, nan, vp).cuda()


def _check(c, oc, want, seed, q_scale=1.0, scale=SCALE, what=""):
    """One attention call of the planned step against the oracle."""
    kp, vp = _fill(c, oc, seed)
    q = (rows_bf16(c.token_cap, c.heads, seed + 2, q_scale)).cuda()
    o, buf, guard = guarded_empty_like(q)
    o.copy_(rows_bf16(c.token_cap, c.heads, seed + 3))
    rest = f64(o)
    c.attn(q, kp, vp, o, softmax_scale=scale)
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    check_guards(buf, guard)
    got = f64(o)
    # scale sum_c |q_c k_c| <= scale |q| |k|
    score_sum = scale * float(q.float().norm(dim=-1).max()
                              * kp.float().nan_to_num().norm(dim=-1).max())
    taken = np.zeros(c.token_cap, bool)
    for r, rows, ref, mag in expect_attn(c, oc, q, kp.nan_to_num(),
                                         vp.nan_to_num(), want, scale):
        assert_attn(got[rows], ref, mag, "%s stream %d" % (what, r),
                    score_sum)
        taken[rows] = True
    assert np.array_equal(got[~taken], rest[~taken]), what
    return q, kp, vp, got


def _run(streams, grid, ps, heads, kv_heads, steps, seed, max_new, n_pages,
         spare=3, check=None, **kw):
    cap = max(sum(max(n, 0) for n in s) for s in steps) + spare
    total = max(s[0] * s[1] for s in streams)
    max_pages = -(-grid[0] * total // ps)
    c, oc = make(streams, grid, n_pages, ps, max_pages, heads, kv_heads, cap,
                 max_new)
    shuffle_ring(c, oc, seed)
    for i, new in enumerate(steps):
        want = step(c, oc, new)
        if check is None or i in check:
            _check(c, oc, want, seed + 10 * i, what="step %d" % i, **kw)
    return c, oc, want


# -------------------------------------------------------------- few rows --

@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 1), (6, 2)])
def test_few_rows_single_tokens(ps, heads, kv_heads):
    # one token from lengths 0, 1, around a page and a stage, ended, idle
    streams = [(2, 2, 1, 0)] * 8
    _run(streams, (100, 2, 2), ps, heads, kv_heads,
         ([1, 2, 2, 1, 1, 0, 1, 1], [1, 1, 2, 0, 1, 2, -1, 1],
          [1, 1, 1, 1, 1, 1, 2, 1]), 50 + ps, 2, 60)


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("kv", [63, 64, 65, 127, 129, 1000])
def test_few_rows_lengths(ps, kv):
    # the cache is filled in steps of at most max_new = 16 rows
    streams = [(4, 4, 16, 0), (4, 4, 1, 0)]
    steps = [[16, 16]] * (kv // 16) + [[kv % 16, kv % 16], [1, 3]]
    _run(streams, (80, 4, 4), ps, 3, 3, steps, kv, 16, 140,
         check=(len(steps) - 1, len(steps) - 2))


@pytest.mark.parametrize("window", [16, 40, 3])
@pytest.mark.parametrize("heads,kv_heads,new", [(1, 1, 16), (4, 2, 7),
                                                (5, 1, 3)])
def test_few_rows_windows_and_chunks(window, heads, kv_heads, new):
    # window 3 is shorter than the chunk: the first rows of a chunk that is
    # only begun see nothing and give 0
    streams = [(4, 4, 16, window), (4, 4, 5, window), (4, 4, 1, window)]
    steps = [[new, new, new]] * 14 + [[1, new, 2]]
    _run(streams, (80, 4, 4), 16, heads, kv_heads, steps, window, new, 100,
         check=(0, 1, 5, 13, 14))


def test_few_rows_peaked_softmax():
    # scores up to about +-60 log2 units: the running maximum moves
    streams = [(8, 8, 1, 0)]
    steps = [[16]] * 40
    _run(streams, (80, 8, 8), 32, 2, 2, steps, 7, 16, 30, check=(39,),
         q_scale=8.0)
