"""GPU parity of the paged cache at sizes where the division of the work
changes: rows sampled from large calls against the formulas in 64 bits on the
same device, and every row checked for having been written."""

import math

import numpy as np
import pytest
import torch

from gpu_common import f64
from paged_common import assert_attn, assert_plan, make, shuffle_ring, step
from test_gpu_paged_attn import _run
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


# -------------------------------------------------- the division of the work

def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# rounds of whole units: a few (their loads are summed, odd rounds run
# backwards), many (the loads count as equal from 16 on)
@pytest.mark.parametrize("R,heads,new_hi,least,most", [
    (8, 40, 600, 2, 5), (20, 32, 560, 5, 12), (30, 72, 500, 16, 40)])
def test_rounds_of_whole_units(R, heads, new_hi, least, most):
    rng = np.random.default_rng(R)
    streams = [(4, 5, int(rng.choice([20, 60])), int(rng.choice([0, 60])))
               for _ in range(R)]
    steps = [[int(x) for x in rng.integers(1, hi + 1, R)]
             for hi in (150, new_hi)]
    units = heads * sum(-(-n // 256) for n in steps[1])
    assert least <= units // _sms() < most
    _run(streams, (60, 4, 5), 64, heads, heads, steps, 40 + R, new_hi,
         R * (2 + (150 + new_hi) // 64) + 20, check=(1,))


def _fill(c, oc, kv):
    """Stream r holds kv[r] positions in pages of its own, in order."""
    at = 0
    for r, n in enumerate(kv):
        held = -(-n // oc.ps)
        c.block_table[r, :held] = torch.arange(at, at + held,
                                               dtype=torch.int32)
        at += held
    assert at <= oc.n_pages
    c.kv_lens.copy_(torch.tensor(kv, dtype=torch.int32))
    c.ring_state.copy_(torch.tensor([at, oc.n_pages - at],
                                    dtype=torch.int32))
    oc.kv = list(kv)


def _plan(c, oc, new):
    """Plans on the device only (the oracle keeps the lengths)."""
    c.plan(torch.tensor(new, dtype=torch.int32, device="cuda"))
    assert c.status.tolist() == [0] * len(new)
    oc.kv = [a + b for a, b in zip(oc.kv, new)]


@pytest.mark.parametrize("heads,streams,new,kv,grid,least", [
    # the 480p chunk of the 12-head model over the cache of 81 frames
    (12, [(30, 52, 4680, 0)], [4680], [28080], (21, 30, 52), 1),
    # four 720p chunks of the 40-head model in one step
    (40, [(45, 80, 10800, 0)] * 4, [10800] * 4, [0, 3600, 7200, 10800],
     (21, 45, 80), 16)])
def test_chunks_of_real_size(heads, streams, new, kv, grid, least):
    cap = sum(new) + 5
    total = [a + b for a, b in zip(new, kv)]
    pages = sum(-(-n // 64) for n in total) + 9
    c, oc = make(streams, grid, pages, 64, -(-max(total) // 64), heads,
                 heads, cap, max(new))
    _fill(c, oc, kv)
    _plan(c, oc, new)
    assert heads * sum(-(-n // 256) for n in new) // _sms() >= least
    kp = _randn((pages, heads, 64, 128), 1)
    vp = _randn((pages, heads, 64, 128), 2)
    q = _randn((cap, heads, 128), 3, 8.0)
    o = _call(c, q, kp, vp)
    assert bool(torch.isfinite(o[:sum(new)]).all())
    assert bool(torch.isnan(o[sum(new):]).all())
    first = 0
    for r, n in enumerate(new):
        _check_rows(c, oc, r, first, _sample(n, 12, r), q, kp, vp, o,
                    "%d heads" % heads)
        first += n


@pytest.mark.parametrize("max_new,new", [(300, [300, 130]), (16, [4, 16])])
def test_a_cache_of_more_than_65535_key_blocks(max_new, new):
    # a stream of 8.5 million positions beside a short one
    kv = [8_500_000, 5000]
    pages = sum(-(-(a + b) // 128) for a, b in zip(kv, new))
    c, oc = make([(100, 100, 1, 0)] * 2, (900, 100, 100), pages, 128, 66500,
                 1, 1, 500, max_new)
    _fill(c, oc, kv)
    _plan(c, oc, new)
    kp = _randn((pages, 1, 128, 128), 1)
    vp = _randn((pages, 1, 128, 128), 2)
    q = _randn((500, 1, 128), 3, 8.0)
    o = _call(c, q, kp, vp)
    assert bool(torch.isfinite(o[:sum(new)]).all())
    assert bool(torch.isnan(o[sum(new):]).all())
    first = 0
    for r, n in enumerate(new):
        _check_rows(c, oc, r, first, _sample(n, 12, r), q, kp, vp, o,
                    "long cache")
        first += n


# ---------------------------------------------------------- the plan's sizes

# 256 threads a CTA for up to 64 streams and 32,768 records, 1,024 beyond; a
# cluster of 8 CTAs up to 32,768 records, of 16 beyond
@pytest.mark.parametrize("R", [1, 64, 65])
@pytest.mark.parametrize("cap", [32768, 32769])
@pytest.mark.parametrize("max_new", [1, 900])
def test_plan_where_its_launch_changes(R, cap, max_new):
    rng = np.random.default_rng(R + cap)
    streams = [(int(rng.integers(1, 6)), int(rng.integers(1, 6)),
                int(rng.integers(1, 40)), int(rng.integers(0, 3) * 37))
               for _ in range(R)]
    c, oc = make(streams, (900, 5, 5), 60 * R + 300, 16, 320, 2, 2, cap,
                 max_new)
    shuffle_ring(c, oc, R)
    for _ in range(4):
        new = rng.integers(-max_new // 8 - 1, max_new + 1, R)
        new[rng.random(R) < 0.2] = 0
        want = step(c, oc, [int(x) for x in new])
        assert_plan(c, oc, want)
