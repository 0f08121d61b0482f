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


# ------------------------------------------------------------- row tiles --

@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 2), (6, 1)])
def test_tiles_ragged_streams(ps, heads, kv_heads):
    # rows around a tile and a tile pair, idle and ended streams, single
    # rows among long ones
    streams = [(4, 5, 20, 0)] * 7
    _run(streams, (60, 4, 5), ps, heads, kv_heads,
         ([17, 1, 128, 129, 0, 256, 257], [300, 127, 1, 20, 255, -1, 3],
          [40, 513, -1, 1, 2, 5, 0]), 500 + ps, 600, 260)


@pytest.mark.parametrize("window,chunk", [
    (0, 1), (0, 20), (40, 20), (7, 20), (300, 60), (130, 1),
    (0, 2 ** 31 - 1)])
def test_tiles_windows_and_chunks(window, chunk):
    streams = [(4, 5, chunk, window), (5, 5, chunk, window)]
    _run(streams, (80, 5, 5), 16, 2, 2,
         ([300, 31], [17, 170], [333, 400], [1, 90]), 700 + window, 400, 220)


@pytest.mark.parametrize("kv", [127, 128, 129, 255, 257, 2000])
def test_tiles_one_row_tile_over_a_cache(kv):
    # the cache first, then 17 rows: ranges of the keys are joined
    streams = [(5, 10, 50, 0)]
    _run(streams, (60, 5, 10), 64, 2, 2, ([kv], [17], [33]), kv, 2000, 40,
         check=(0, 1, 2))


def test_tiles_many_units_per_cta():
    # several units a CTA in every mix of one and two tiles, none visible
    streams = [(4, 5, 20, 0 if i % 3 else 3) for i in range(40)]
    new0 = [7 * i % 290 + 1 for i in range(40)]
    new1 = [11 * i % 270 for i in range(40)]
    _run(streams, (60, 4, 5), 32, 8, 4, (new0, new1), 900, 300, 900)


def test_tiles_peaked_softmax():
    streams = [(8, 8, 64, 0)]
    _run(streams, (60, 8, 8), 32, 2, 2, ([700], [500]), 31, 700, 40,
         q_scale=8.0)


def test_tiles_first_keys_hidden_from_some_rows():
    # rows of one warp whose first block holds no visible key beside rows
    # whose maximum moves by more than 2^8 a block later
    streams = [(2, 2, 4, 150)]
    _run(streams, (400, 2, 2), 16, 1, 1, ([900], [400]), 41, 900, 90,
         q_scale=8.0)


# --------------------------------------------------------- both kernels --

@pytest.mark.parametrize("max_new", [16, 200])
def test_pages_out_of_range_read_as_zero(max_new):
    c, oc = make([(4, 4, 16, 0)], (20, 4, 4), 12, 16, 20, 1, 1, 16, max_new)
    for new in ([16], [16], [16], [10]):
        want = step(c, oc, new)
    kp, vp = _fill(c, oc, 5)
    kp, vp = kp.nan_to_num(), vp.nan_to_num()
    q = rows_bf16(16, 1, 9).cuda()
    o = torch.zeros_like(q)
    for bad in (-1, 12, 2 ** 31 - 1, -2 ** 31):
        c.block_table[0, 1] = bad
        c.attn(q, kp, vp, o)
        torch.cuda.synchronize()
        kz, vz = kp.clone(), vp.clone()
        kz[oc.table[0][1]] = 0
        vz[oc.table[0][1]] = 0
        (_, rows, ref, mag), = expect_attn(c, oc, q, kz, vz, want, SCALE)
        assert_attn(f64(o)[rows], ref, mag, "page %d" % bad, 30.0)


@pytest.mark.parametrize("max_new,new", [(4, 4), (700, 700)])
def test_same_result_every_time_and_in_a_graph(max_new, new):
    streams = [(8, 8, 64, 0)] * 3
    cap = 3 * 700
    c, oc = make(streams, (60, 8, 8), 200, 32, 60, 2, 2, cap, 700)
    step(c, oc, [700, 650, 10])
    c.max_new = max_new
    lens = torch.tensor([new, max(1, new // 3), 1], dtype=torch.int32,
                        device="cuda")
    kp, vp = c.new_pools()
    kp.normal_()
    vp.normal_()
    q = rows_bf16(cap, 2, 9).cuda()
    o = torch.zeros_like(q)
    saved = c.state.clone()
    c.plan(lens)
    c.attn(q, kp, vp, o)
    first = o.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.plan(lens)
        c.attn(q, kp, vp, o)
    for _ in range(3):
        c.state.copy_(saved)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)
    # other lengths through the same graph
    lens.copy_(torch.tensor([1, 2, 3], dtype=torch.int32))
    c.state.copy_(saved)
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = o.clone()
    want = oc.plan([1, 2, 3])
    for _, rows, ref, mag in expect_attn(c, oc, q, kp, vp, want, SCALE):
        assert_attn(f64(got)[rows], ref, mag, "replay", 30.0)


def test_a_graph_keeps_its_workspace_when_max_new_grows():
    """A captured single-token step goes on using the scratch it was captured
    with after steps that need more: what is allocated later stays whole."""
    streams = [(8, 8, 64, 0)] * 2
    cap = 32
    c, oc = make(streams, (60, 8, 8), 100, 32, 60, 2, 2, cap, 16)
    for _ in range(12):                    # three key stages a stream
        step(c, oc, [16, 15])
    kp, vp = c.new_pools()
    kp.normal_()
    vp.normal_()
    q = rows_bf16(cap, 2, 11).cuda()
    o = torch.zeros_like(q)
    small = c.workspace()
    size = small.numel()
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    saved = c.state.clone()
    c.plan(lens)
    c.attn(q, kp, vp, o)
    first = o.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.plan(lens)
        c.attn(q, kp, vp, o)
    at = small.data_ptr()
    del small
    c.max_new = 700
    assert c.workspace().numel() > size
    later = [torch.full((size,), 77, dtype=torch.uint8, device="cuda")
             for _ in range(4)]
    c.state.copy_(saved)
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, first)
    for t in later:
        assert bool((t == 77).all())
    c.max_new = 16
    assert c.workspace().data_ptr() == at


def test_write_and_attention_over_layers_match_the_whole_video():
    """Three chunks of a video through plan, write and attention of two
    layers give what the contiguous calls give on the whole video."""
    grid, heads, chunk = (6, 4, 5), 2, 40
    L = 120
    g = wan.grid(*grid)
    table = wan.rope3d_table(g)
    c, oc = make([(4, 5, chunk, 0)], grid, 9, 16, 9, heads, heads, chunk)
    kp, vp = c.new_pools(2)
    w = torch.rand(heads * 128, device="cuda") + 0.5
    qkv = [[rows_bf16(L, heads, 60 + 3 * i + j).cuda() for j in range(3)]
           for i in range(2)]
    outs = [torch.zeros(L, heads, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    for i in range(3):
        step(c, oc, [chunk])
        part = slice(chunk * i, chunk * (i + 1))
        for layer in range(2):
            q, k, v = (x[part].clone() for x in qkv[layer])
            c.write(q, k, v, w, w, table, kp[layer], vp[layer])
            o = torch.empty_like(q)
            c.attn(q, kp[layer], vp[layer], o)
            outs[layer][part] = o
    for layer in range(2):
        q, k, v = (x.clone()[None] for x in qkv[layer])
        wan.qk_norm_rope(q, k, w, w, g, table)
        o = torch.empty_like(q)
        wan.block_causal_attn(q, k, v, o, chunk)
        torch.cuda.synchronize()
        # two kernels, each within its bound of the exact value
        a, b = f64(outs[layer]), f64(o[0])
        mag = np.abs(f64(v)).max()
        assert np.max(np.abs(a - b)) <= 2 * (2 ** -7 + 1e-3) * mag
        assert np.linalg.norm(a - b) <= 1e-2 * np.linalg.norm(b)


def test_class_refuses_tensors_that_do_not_fit():
    c, oc = make([(4, 4, 16, 0)], (20, 4, 4), 12, 16, 20, 4, 2, 16)
    kp, vp = c.new_pools()
    q = rows_bf16(16, 4, 1).cuda()
    k, v = rows_bf16(16, 2, 2).cuda(), rows_bf16(16, 2, 3).cuda()
    o = torch.empty_like(q)
    w4, w2 = torch.ones(512, device="cuda"), torch.ones(256, device="cuda")
    table = wan.rope3d_table(c.grid)
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="plan"):
        c.attn(q, kp, vp, o)
    for bad in (lens.long(), lens.cpu(), lens[:0], lens.repeat(2)):
        with pytest.raises(ValueError):
            c.plan(bad)
    c.plan(lens)
    good = dict(q=q, k=k, v=v, wq=w4, wk=w2, table=table, k_pages=kp,
                v_pages=vp)
    for name, t in good.items():
        bads = [t.cpu(), t[:-1]]
        if t.dtype != torch.uint8:
            bads.append(t.double())
        for bad in bads:
            with pytest.raises(ValueError):
                c.write(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        c.write(**good, q_out=o[:-1])
    with pytest.raises(ValueError):
        c.write(**dict(good, table=None))
    for args in ((q[:-1], kp, vp, o), (q, kp[:-1], vp, o), (q, kp, vp, o[1:]),
                 (q.float(), kp, vp, o), (q, kp, vp.cpu(), o),
                 (q.transpose(0, 1), kp, vp, o)):
        with pytest.raises(ValueError):
            c.attn(*args)
    with pytest.raises(ValueError, match="bytes"):
        c.attn(q, kp, vp, o, workspace=torch.empty(16, dtype=torch.uint8,
                                                   device="cuda"))
    with pytest.raises(wan.WanError):
        c.attn(q, kp, vp, o, softmax_scale=-1.0)
    with pytest.raises(wan.WanError):
        c.attn(q, kp, vp, q)
    c.max_new = 2                      # another kernel than the plan's
    with pytest.raises(ValueError, match="max_new"):
        c.attn(q, kp, vp, o)


def test_two_calls_at_once_with_a_workspace_each():
    streams = [(8, 8, 64, 0)] * 2
    c, oc = make(streams, (60, 8, 8), 160, 32, 60, 2, 2, 1400, 700)
    step(c, oc, [700, 650])
    kp, vp = c.new_pools(2)
    kp.normal_()
    vp.normal_()
    q = [rows_bf16(1400, 2, 9 + i).cuda() for i in range(2)]
    want, o = [], [torch.zeros_like(q[0]) for _ in range(2)]
    for i in range(2):
        c.attn(q[i], kp[i], vp[i], o[i])
        torch.cuda.synchronize()
        want.append(o[i].clone())
        o[i].zero_()
    ws = [torch.empty(c.workspace_bytes(), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            c.attn(q[i], kp[i], vp[i], o[i], stream=side[i],
                   workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(o[i], want[i])


@pytest.mark.parametrize("seed", range(12))
def test_random_streams(seed):
    """Seeded shapes of both kernels: streams, windows, chunks, heads, page
    sizes, lengths; three steps each, every one checked."""
    rng = np.random.default_rng(1000 + seed)
    few = seed % 2 == 0
    kv_heads = int(rng.integers(1, 4))
    group = int(rng.integers(1, 5))
    R = int(rng.integers(1, 7))
    ps = int(rng.choice([16, 32, 64, 128]))
    max_new = max(1, int(rng.integers(1, 17)) // group) if few \
        else int(rng.integers(17, 420))
    streams = [(4, 5, int(rng.choice([1, 7, 20, 60, 10 ** 9])),
                int(rng.choice([0, 0, 5, 33, 100, 400]))) for _ in range(R)]
    steps = []
    for _ in range(8 if few else 3):
        new = rng.integers(0, max_new + 1, R)
        new[rng.random(R) < 0.1] = -1
        steps.append([int(x) for x in new])
    _run(streams, (400, 4, 5), ps, kv_heads * group, kv_heads, steps,
         3000 + seed, max_new, 40 * R + 100,
         check=(1, len(steps) - 2, len(steps) - 1))


@pytest.mark.parametrize("max_new", [16, 300])
def test_pools_past_32_bit_offsets(max_new):
    # K and V pools of 2.3e9 elements each, the stream's pages at their end
    # (and one at the front)
    ps, kv_heads, n_pages = 128, 8, 17600
    assert n_pages * ps * kv_heads * 128 > 2 ** 31
    c, oc = make([(8, 8, 64, 0)], (20, 8, 8), n_pages, ps, 10, 8, kv_heads,
                 300, max_new)
    oc.ring = [n_pages - 1, 0] + list(range(n_pages - 2, 0, -1))
    c.free_ring.copy_(torch.tensor(oc.ring, dtype=torch.int32))
    kp, vp = c.new_pools()
    w = torch.ones(kv_heads * 128, device="cuda")
    table = wan.rope3d_table(c.grid)
    keys = torch.zeros(0, kv_heads, 128, dtype=torch.bfloat16)
    vals = keys
    for i, n in enumerate([max_new] * (320 // max_new) + [7]):
        want = step(c, oc, [n])
        q, k, v = (rows_bf16(300, 8, 40 + 3 * i + j).cuda() for j in range(3))
        c.write(q, k, v, w, w, table, kp, vp)
        o = torch.zeros_like(q)
        c.attn(q, kp, vp, o)
        slots = c.tokens[:n, 3].cpu().long()
        assert int(slots.max()) >= (n_pages - 9) * ps or int(
            slots.max()) < 128
        page, off = slots.cuda() // ps, slots.cuda() % ps
        keys = torch.cat([keys, kp[page, :, off].cpu()])
        vals = torch.cat([vals, vp[page, :, off].cpu()])
        assert torch.equal(vals[-n:], v[:n].cpu())
    torch.cuda.synchronize()
    s = np.einsum("ihd,jhd->hij", f64(q)[:7], f64(keys)) * SCALE
    a = np.arange(oc.kv[0] - 7, oc.kv[0])[:, None]
    j = np.arange(oc.kv[0])[None]
    s = np.where(j < (a // 64 + 1) * 64, s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref = np.einsum("hij,jhd->ihd", p, f64(vals))
    mag = np.einsum("hij,jhd->ihd", p, np.abs(f64(vals)))
    assert_attn(f64(o)[:7], ref, mag, "large pool", 40.0)


@pytest.mark.parametrize("R,max_new", [(33, 2), (100, 1), (1024, 3),
                                       (70, 130)])
def test_many_streams(R, max_new):
    # work lists past one warp's width: searched in memory
    rng = np.random.default_rng(R)
    streams = [(2, 3, int(rng.choice([1, 6])), int(rng.choice([0, 12])))
               for _ in range(R)]
    steps = [[int(x) for x in rng.integers(0, max_new + 1, R)]
             for _ in range(4)]
    _run(streams, (200, 2, 3), 16, 2, 1, steps, 77 + R, max_new,
         R * (1 + 4 * max_new // 16) + R + 20, check=(0, 3))


# head groups of a row tile: all heads of one key head, a divisor of them, one
# (a prime past 16), and long streams whose tiles would not come out even
@pytest.mark.parametrize("heads,kv_heads,max_new", [
    (5, 1, 300), (16, 1, 300), (20, 1, 200), (17, 1, 100), (32, 1, 100),
    (14, 2, 300), (5, 1, 1100), (8, 2, 1100)])
def test_tiles_head_groups(heads, kv_heads, max_new):
    streams = [(4, 5, 20, 0), (4, 5, 7, 50), (4, 5, 1, 0)]
    m = max_new
    _run(streams, (130, 4, 5), 16, heads, kv_heads,
         ([m, 1, 26], [25, m, 127], [51, 130, 3]), 60 + heads, m,
         3 * (2 * m + 200) // 16 + 40)
