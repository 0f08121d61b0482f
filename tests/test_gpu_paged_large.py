"""GPU parity of the paged cache at sizes where the division of the work
changes: rows sampled from large calls against the formulas in 64 bits on the
same device, and every row checked for having been written."""

import math

import numpy as np
import pytest
import torch

from gpu_common import f64
from paged_common import assert_attn, make, step
from video_diffusion_transformer_self_b200 import build, wan

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wan.lib()


def _randn(shape, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):     # fp32 draws, by parts
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda") * scale
    return out


def _call(c, q, kp, vp):
    """One attention call into an output of NaN."""
    o = torch.full_like(q, float("nan"))
    c.attn(q, kp, vp, o)
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    return o


def _check_rows(c, oc, r, first, rows, q, kp, vp, o, what):
    """Rows (offsets in stream r, whose packed rows start at first) against
    64 bits; the queries are scaled so that few keys carry a row and another
    row's result would not pass."""
    chunk, window = oc.streams[r][2:]
    kv, ps = oc.kv[r], oc.ps
    n = int(c.q_lens[r])
    lo_all = 0 if not window else max(
        0, ((kv - n) // chunk + 1) * chunk - window)
    j = torch.arange(lo_all, kv, device="cuda")
    page = c.block_table[r].long()[j // ps]
    group = c.heads // c.kv_heads
    for h in range(c.heads):
        if h % group == 0:
            k = kp[page, h // group, j % ps].double()
            v = vp[page, h // group, j % ps].double()
        for i in rows:
            a = kv - n + i
            e = (a // chunk + 1) * chunk
            lo = max(0, e - window) if window else 0
            kk = k[lo - lo_all:min(kv, e) - lo_all]
            vv = v[lo - lo_all:min(kv, e) - lo_all]
            qr = q[first + i, h].double()
            if kk.shape[0] == 0:
                assert not o[first + i, h].any(), (what, r, i, h)
                continue
            p = torch.softmax(kk @ qr * SCALE, 0)
            score_sum = SCALE * float(qr.norm() * kk.norm(dim=1).max())
            assert_attn(f64(o[first + i, h]), (p @ vv).cpu().numpy(),
                        (p @ vv.abs()).cpu().numpy(),
                        "%s stream %d row %d head %d" % (what, r, i, h),
                        score_sum)


def _sample(n, count, seed):
    rng = np.random.default_rng(seed)
    picks = {0, n - 1, min(n - 1, 127), min(n - 1, 128), n // 2}
    picks.update(int(x) for x in rng.integers(0, n, count))
    return sorted(picks)


def test_a_million_tokens_of_shared_heads():
    # the weights of one head group's units pass 2^32.  (The softmax is
    # peaked: a few of the 2^20 keys carry a row, so the running sums see
    # little of the others and the bound for short ones holds.)
    T = (1 << 20) + 17
    c, oc = make([(1024, 1024, 1, 0)], (2, 1024, 1024), 8200, 128, 8200, 16,
                 1, T)
    step(c, oc, [T])
    kp, vp = _randn((8200, 1, 128, 128), 1), _randn((8200, 1, 128, 128), 2)
    q = _randn((T, 16, 128), 3, 8.0)
    o = _call(c, q, kp, vp)
    assert bool(torch.isfinite(o).all())
    _check_rows(c, oc, 0, 0, _sample(T, 40, 4), q, kp, vp, o, "2^20 tokens")
