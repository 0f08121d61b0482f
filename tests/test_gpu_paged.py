"""GPU parity of the paged cache's plan and write against the oracle."""

import numpy as np
import pytest
import torch

from gpu_common import check_guards, cuda, f64, guarded_empty_like
from oracle import paged as opaged
from paged_common import (assert_plan, assert_write, make, rows_bf16,
                          shuffle_ring, step)
from video_diffusion_transformer_self_b200 import build, inputs, wan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wan.lib()


# ------------------------------------------------------------------ plan --

@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 24, 5])
def test_plan_steps_of_three_streams(ps, window):
    # grow, idle, end and restart over several steps; window 24 is two
    # chunks of 12, 5 less than one chunk
    streams = [(3, 4, 12, window), (3, 4, 12, 0), (2, 3, 1, window)]
    c, oc = make(streams, (64, 3, 4), 60, ps, 40, 2, 2, 150)
    shuffle_ring(c, oc, 5)
    for i, new in enumerate(([12, 0, 1], [12, 5, 1], [7, 100, 0],
                             [5, -1, 30], [0, 1, -1], [36, 12, 6],
                             [-1, 0, 0], [1, -1, 17])):
        want = step(c, oc, new)
        assert_plan(c, oc, want, "step %d" % i)
    held = sum(p >= 0 for row in oc.table for p in row)
    assert held + oc.count == oc.n_pages


def test_plan_refuses_what_does_not_fit():
    # max_pages, grid, max_new, token_cap, settings; the others go on
    streams = [(2, 2, 4, 0), (2, 2, 4, 0), (2, 2, 4, 0), (5, 2, 4, 0),
               (2, 2, 0, 0), (2, 2, 4, -1), (2, 2, 4, 0), (2, 2, 4, 0)]
    c, oc = make(streams, (8, 4, 4), 50, 16, 2, 2, 2, 90, max_new=33)
    for new in ([32, 33, 34, 4, 4, 4, 1, 20], [1, 20, 0, 0, 0, 0, 31, 13],
                [0, 0, 0, 0, 0, 0, 1, 0], [-1, -1, -1, -1, -1, -1, -1, -1]):
        want = step(c, oc, new)
        assert_plan(c, oc, want, str(new))
    assert oc.count == oc.n_pages
    # the last stream's rows pass token_cap
    want = step(c, oc, [30, 30, 0, 0, 0, 0, 30, 1])
    assert want[2][7] == opaged.EINVAL
    assert_plan(c, oc, want, "token_cap")


def test_plan_stops_at_the_first_that_lacks_pages():
    streams = [(4, 4, 16, 0)] * 5
    c, oc = make(streams, (64, 4, 4), 7, 16, 20, 2, 2, 400)
    want = step(c, oc, [48, 48, 33, 1, 0])
    assert want[2] == [0, 0, opaged.ENOSPACE, opaged.ENOSPACE, 0]
    assert_plan(c, oc, want)
    # pages of an ended stream serve the same step; no overtaking
    want = step(c, oc, [-1, 0, 33, 17, 1])
    assert want[2] == [0, 0, 0, opaged.ENOSPACE, opaged.ENOSPACE]
    assert_plan(c, oc, want)
    # a row inside a held page needs no page
    want = step(c, oc, [0, 0, 1, 16, 0])
    assert_plan(c, oc, want)


# one stream to the most, a record to tens of thousands
@pytest.mark.parametrize("R,cap,hi,seed", [
    (1, 1, 1, 0), (1, 5000, 5000, 1), (33, 2048, 90, 2), (33, 2049, 90, 3),
    (1000, 9000, 20, 4), (1024, 40000, 60, 5), (1024, 2000, 3, 6)])
def test_plan_random(R, cap, hi, seed):
    rng = np.random.default_rng(seed)
    streams = [(int(rng.integers(1, 6)), int(rng.integers(1, 6)),
                int(rng.integers(1, 40)), int(rng.integers(0, 3) * 37))
               for _ in range(R)]
    c, oc = make(streams, (900, 5, 5), 4 * R + 300, 16, 320, 2, 1, cap)
    shuffle_ring(c, oc, seed)
    for _ in range(5):
        new = rng.integers(-hi // 8 - 1, hi + 1, R)
        new[rng.random(R) < 0.2] = 0
        want = step(c, oc, [int(x) for x in new])
        assert_plan(c, oc, want)


def test_plan_saved_state_and_graph():
    streams = [(3, 4, 12, 24)] * 6
    c, oc = make(streams, (64, 3, 4), 90, 16, 40, 2, 2, 300)
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    c.plan(lens)                       # first launch outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.plan(lens)
    for new in ([12, 1, 0, 50, 9, 3], [12, 1, 4, 50, -1, 3]):
        saved = c.state.clone()
        for again in range(2):
            c.state.copy_(saved)
            lens.copy_(torch.tensor(new, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
        assert_plan(c, oc, oc.plan(new))


# ----------------------------------------------------------------- write --

def _write_case(heads, kv_heads, ps, streams, grid, steps, spare, seed,
                in_place=False):
    cap = max(sum(max(n, 0) for n in s) for s in steps) + spare
    c, oc = make(streams, grid, 40, ps, 30, heads, kv_heads, cap)
    shuffle_ring(c, oc, seed)
    kp = inputs.randn_bf16((40, kv_heads, ps, 128), seed + 1).cuda()
    vp = inputs.randn_bf16((40, kv_heads, ps, 128), seed + 2).cuda()
    wq = inputs.randn_f32((heads * 128,), seed + 3)
    wk = inputs.randn_f32((kv_heads * 128,), seed + 4)
    table = wan.rope3d_table(wan.grid(*grid))
    for i, new in enumerate(steps):
        want = step(c, oc, new)
        q = rows_bf16(cap, heads, seed + 10 + i, 2.0)
        k = rows_bf16(cap, kv_heads, seed + 20 + i, 0.5)
        v = rows_bf16(cap, kv_heads, seed + 30 + i)
        kp0, vp0 = f64(kp), f64(vp)
        qg, kg, vg = cuda(q), cuda(k), cuda(v)
        if in_place:
            out = qg
            rest = f64(qg)
            c.write(qg, kg, vg, cuda(wq), cuda(wk), table, kp, vp)
        else:
            out, buf, guard = guarded_empty_like(qg)
            out.copy_(rows_bf16(cap, heads, seed + 40 + i))
            rest = f64(out)
            c.write(qg, kg, vg, cuda(wq), cuda(wk), table, kp, vp, q_out=out)
            check_guards(buf, guard)
            assert torch.equal(qg.cpu(), q)
        torch.cuda.synchronize()
        assert torch.equal(kg.cpu(), k) and torch.equal(vg.cpu(), v)
        rec = np.asarray(want[3])
        live = np.nonzero(rec[:, 3] >= 0)[0]
        dead = np.nonzero(rec[:, 3] < 0)[0]
        assert np.array_equal(f64(out)[dead], rest[dead])
        pos, slot = rec[live, :3], rec[live, 3]
        kn, vn = kp0, vp0
        for name, x, w in (("q", q, wq), ("k", k, wk)):
            x64, w64 = f64(x)[live], w.double().numpy()
            ref = opaged.norm_rope_rows(x64, w64, pos)
            y = opaged.norm_rope_rows(x64, w64, np.zeros_like(pos))
            mag = np.repeat(np.abs(y[..., 0::2]) + np.abs(y[..., 1::2]), 2,
                            axis=-1)
            if name == "q":
                assert_write(f64(out)[live], ref, mag, "q")
            else:
                got = f64(kp)[slot // ps, :, slot % ps]
                assert_write(got, ref, mag, "k")
                kn[slot // ps, :, slot % ps] = got
        vn[slot // ps, :, slot % ps] = f64(v)[live]
        # nothing else of the pools was touched, v is copied bit by bit
        assert np.array_equal(f64(kp), kn)
        assert np.array_equal(f64(vp), vn)


# heads across the register variants (4, 6, 8, 12, 20 rows a lane) and the
# two-pass one, shared key heads, odd counts
@pytest.mark.parametrize("heads,kv_heads", [
    (1, 1), (2, 2), (7, 7), (8, 2), (9, 3), (12, 12), (13, 1), (16, 1),
    (17, 17),
    (25, 5), (40, 40), (40, 8), (41, 41), (48, 6)])
def test_write_heads(heads, kv_heads):
    _write_case(heads, kv_heads, 32, [(3, 4, 12, 0), (2, 5, 10, 0)],
                (20, 3, 5), ([5, 12], [30, 0], [1, 1]), 3, 100 + heads)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_write_pages_windows_and_refusals(ps, in_place):
    # a refused stream in the middle, an evicting one, one that ends
    streams = [(3, 4, 12, 24), (9, 9, 12, 0), (2, 5, 1, 7), (1, 1, 1, 0)]
    _write_case(4, 2, ps, streams, (40, 4, 5),
                ([24, 6, 17, 1], [12, 6, 0, 1], [36, 0, 40, 0],
                 [1, 1, -1, 3]), 5, 300, in_place)


def test_write_ignores_records_no_plan_writes():
    c, oc = make([(3, 4, 12, 0)], (5, 3, 4), 6, 16, 6, 2, 2, 9)
    step(c, oc, [9])
    base = c.tokens.clone()
    bad = [(0, 0, 0, 96), (0, 0, 0, 2 ** 31 - 1), (0, 0, 0, -7),
           (5, 0, 0, 0), (-1, 0, 0, 1), (0, 3, 0, 2), (0, -1, 0, 3),
           (0, 0, 4, 4), (2 ** 31 - 1, -2 ** 31, 2 ** 30, 5)]
    c.tokens.copy_(torch.tensor(bad, dtype=torch.int32))
    kp, vp = c.new_pools()
    q = cuda(rows_bf16(9, 2, 1))
    k, v = cuda(rows_bf16(9, 2, 2)), cuda(rows_bf16(9, 2, 3))
    w = torch.ones(256, device="cuda")
    q0 = q.clone()
    c.write(q, k, v, w, w, wan.rope3d_table(c.grid), kp, vp)
    torch.cuda.synchronize()
    assert torch.equal(q, q0)
    assert not kp.any() and not vp.any()
    c.tokens.copy_(base)
    c.write(q, k, v, w, w, wan.rope3d_table(c.grid), kp, vp)
    torch.cuda.synchronize()
    assert not torch.equal(q, q0) and kp.any() and vp.any()
