"""What the paged cache does around a step: plans that do not belong to the
attention call, scratch on other streams, values that are not finite."""

import math

import numpy as np
import pytest
import torch

from gpu_common import f64
from paged_common import (assert_attn, expect_attn, make, rows_bf16, step)
from video_diffusion_transformer_self_b200 import build, wan

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wan.lib()


# the kernel, the rows of a key head, the heads of a row tile (5 heads share a
# tile up to max_new 1,024), each way round
@pytest.mark.parametrize("heads,kv_heads,graph_max,call_max", [
    (2, 2, 700, 16), (2, 2, 16, 700), (2, 2, 16, 2), (2, 2, 2, 16),
    (5, 1, 1100, 300), (5, 1, 300, 1100), (8, 1, 1100, 300)])
def test_attention_refuses_a_plan_replayed_with_another_max_new(
        heads, kv_heads, graph_max, call_max):
    c, oc = make([(8, 8, 64, 0)] * 2, (60, 8, 8), 60, 32, 40, heads, kv_heads,
                 64, graph_max)
    lens = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    kp, vp = c.new_pools()
    kp.normal_()
    vp.normal_()
    q = rows_bf16(64, heads, 5).cuda()
    o = rows_bf16(64, heads, 6).cuda()
    rest = o.clone()
    saved = c.state.clone()
    c.plan(lens)                     # first launches outside the capture
    c.state.copy_(saved)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.plan(lens)
    c.max_new = call_max
    c.plan(lens)                     # what the class remembers
    oc.plan([2, 1])
    c.attn(q, kp, vp, torch.zeros_like(o))
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    graph.replay()
    want = oc.plan([2, 1])
    c.attn(q, kp, vp, o)
    torch.cuda.synchronize()
    same = (heads, kv_heads) == (8, 1)   # 8 heads share a tile either way
    assert wan.device_status() == (0 if same else wan.WAN_EINVAL)
    assert wan.device_status() == 0      # read and cleared
    if same:
        for _, rows, ref, mag in expect_attn(c, oc, q, kp, vp, want, SCALE):
            assert_attn(f64(o)[rows], ref, mag, "same layout", 30.0)
        return
    assert torch.equal(o, rest)
    # a plan of the call's own kind serves it again
    c.plan(lens)
    want = oc.plan([2, 1])
    c.attn(q, kp, vp, o)
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    for _, rows, ref, mag in expect_attn(c, oc, q, kp, vp, want, SCALE):
        assert_attn(f64(o)[rows], ref, mag, "planned again", 30.0)
    taken = np.zeros(64, bool)
    taken[:3] = True
    assert np.array_equal(f64(o)[~taken], f64(rest)[~taken])


def test_no_call_allocates_whatever_max_new_becomes():
    """Scratch of both kernels exists before the first call: none is taken
    from the current stream's memory for a call on another stream."""
    for first, heads, kv_heads in ((16, 2, 2), (700, 2, 2), (1, 40, 2)):
        c, oc = make([(8, 8, 64, 0)] * 2, (60, 8, 8), 60, 32, 40, heads,
                     kv_heads, 64, first)
        kp, vp = c.new_pools()
        q = rows_bf16(64, heads, 5).cuda()
        o = torch.zeros_like(q)
        lens = torch.ones(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        for max_new in (first, 700, 16, 1, 3000, 64, 10 ** 9):
            c.max_new = max_new
            c.plan(lens, stream=side)
            c.attn(q, kp, vp, o, stream=side)
            assert c.workspace().numel() == c.workspace_bytes() > 0
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        torch.cuda.synchronize()
        assert wan.device_status() == 0


# one part a row and many (few keys, many keys), both kernels
@pytest.mark.parametrize("max_new", [4, 300])
@pytest.mark.parametrize("kv", [30, 5000])
def test_rows_that_are_not_finite_stay_so_however_they_are_cut(max_new, kv):
    """A NaN or infinity in a query gives NaN in its row and in no other,
    whether one CTA has the row's keys or the partial results of many are
    joined; a NaN key gives NaN in the rows of the few-row kernel that see
    it."""
    n = 4
    c, oc = make([(10, 10, 1, 0)], (60, 10, 10), 330, 16, 330, 2, 2, n,
                 max_new)
    c.max_new = max_new
    c.kv_lens[0] = oc.kv[0] = kv
    held = -(-kv // 16)
    pages = list(range(held))
    c.block_table[0, :held] = torch.arange(held, dtype=torch.int32)
    oc.table[0][:held] = pages
    c.ring_state.copy_(torch.tensor([held, 330 - held], dtype=torch.int32))
    oc.head, oc.count = held, 330 - held
    want = step(c, oc, [n])
    kp, vp = c.new_pools()
    kp.normal_()
    vp.normal_()
    q = rows_bf16(n, 2, 5).cuda()
    o = torch.zeros_like(q)
    for bad in (float("nan"), float("inf"), -float("inf")):
        qb = q.clone()
        qb[1, 0, 7] = bad
        c.attn(qb, kp, vp, o)
        torch.cuda.synchronize()
        assert bool(torch.isnan(o[1, 0]).all()), bad
        good = torch.ones(n, 2, dtype=torch.bool)
        good[1, 0] = False
        (_, rows, ref, mag), = expect_attn(c, oc, q, kp, vp, want, SCALE)
        got = f64(o)[rows]
        keep = good.numpy()
        assert_attn(got[keep], ref[keep], mag[keep], "others", 40.0)
    if max_new == 4:
        at = kv + 2                  # the third row's own position
        kp[oc.table[0][at // 16], 1, at % 16, 3] = float("nan")
        c.attn(q, kp, vp, o)
        torch.cuda.synchronize()
        nan = torch.isnan(o).all(-1).cpu()
        assert nan.tolist() == [[False, False], [False, False],
                                [False, True], [False, True]]
        assert bool(torch.isfinite(o[~nan.cuda()]).all())
    assert wan.device_status() == 0


@pytest.mark.parametrize("max_new", [2 ** 31, 2 ** 32 + 5, 10 ** 18])
def test_max_new_past_32_bits_is_no_limit(max_new):
    c, oc = make([(8, 8, 64, 0)], (60, 8, 8), 60, 32, 40, 2, 2, 300, max_new)
    want = step(c, oc, [300])
    assert c.status.tolist() == [0] and c.q_lens.tolist() == [300]
    kp, vp = c.new_pools()
    kp.normal_()
    vp.normal_()
    q = rows_bf16(300, 2, 5).cuda()
    o = torch.zeros_like(q)
    c.attn(q, kp, vp, o)
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    (_, rows, ref, mag), = expect_attn(c, oc, q, kp, vp, want, SCALE)
    assert_attn(f64(o)[rows], ref, mag, "max_new %d" % max_new, 30.0)


@pytest.mark.parametrize("max_new,steps", [
    (16, [[5, 17, 16, 0, 1], [16, 3, 30, 2, -1], [1, 16, 0, 40, 9]]),
    (300, [[30, 301, 129, 0, 1], [257, 3, 400, 300, -1],
           [300, 16, 0, 333, 90]])])
def test_rows_of_no_stream_may_hold_anything(max_new, steps):
    """Streams refused in the middle of the packing and rows behind the last
    one, all NaN: the others' results are whole, theirs stay as they were."""
    cap = max(sum(max(n, 0) for n in s) for s in steps) + 9
    c, oc = make([(8, 8, 64, 0), (8, 8, 1, 100)] * 2 + [(8, 8, 20, 30)],
                 (60, 8, 8), 200, 16, 70, 4, 2, cap, max_new)
    kp, vp = c.new_pools()
    w4, w2 = torch.ones(512, device="cuda"), torch.ones(256, device="cuda")
    table = wan.rope3d_table(c.grid)
    for i, new in enumerate(steps):
        want = step(c, oc, new)
        assert any(s == wan.WAN_EINVAL for s in want[2])
        taken = torch.zeros(cap, dtype=torch.bool)
        for at, n in zip(want[0], want[1]):
            taken[at:at + n] = True
        q, k, v = (rows_bf16(cap, h, 10 * i + j)
                   for j, h in enumerate((4, 2, 2)))
        for t in (q, k, v):
            t[~taken] = float("nan")
        q, k, v = q.cuda(), k.cuda(), v.cuda()
        c.write(q, k, v, w4, w2, table, kp, vp)
        o = rows_bf16(cap, 4, 10 * i + 5).cuda()
        rest = o.clone()
        c.attn(q, kp, vp, o)
        torch.cuda.synchronize()
        assert wan.device_status() == 0
        assert bool(torch.isfinite(kp).all() and torch.isfinite(vp).all())
        assert torch.equal(torch.isnan(q).all(-1).all(-1).cpu(), ~taken)
        assert torch.equal(o[~taken.cuda()], rest[~taken.cuda()])
        for r, rows, ref, mag in expect_attn(c, oc, q, kp, vp, want, SCALE):
            assert_attn(f64(o)[rows], ref, mag, "step %d stream %d" % (i, r),
                        40.0)
