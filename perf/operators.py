"""Cases and plain forms of the paged K/V cache: the plan of a step (block
tables, slots and positions from the streams' lengths), the write of the new
tokens (QK-Norm, RoPE of each token's time / height / width position, K and V
into their pages) and the chunk-causal attention over the pages.

``own`` false computes the operators with elementary torch operations,
``own`` true calls the framework's kernels.
"""

import math
import random

import torch

own = False

HD = 128
EPS = 1e-6
THETA = 10000.0
DEV = "cuda"


# ------------------------------------------------------------------ cases --

def _case(name, op, **kw):
    c = dict(name=name, op=op, layout=1, streams=1, heads=12, kv_heads=12,
             page=64, frame_h=30, frame_w=52, chunk=4680, window=0, new_lo=1,
             new_hi=1, kv_lo=0, kv_hi=0, whole=False, ended=0, idle=0,
             tight=False, spare=0)
    c.update(kw)
    return c


def listed():
    return [
        # one 480p stream takes its next chunk of three latent frames
        _case("plan-1x4680", "plan", new_lo=4680, new_hi=4680, kv_lo=28080,
              kv_hi=28080, whole=True, window=65520, spare=5),
        # a server of 48 streams: ended and idle ones, caches capped at 42
        # latent frames, pages of 16 tokens
        _case("plan-48-capped", "plan", streams=48, layout=2, page=16,
              new_lo=1560, new_hi=4680, kv_lo=1560, kv_hi=93600, whole=True,
              window=65520, ended=7, idle=5, spare=129),
        # 777 short requests, one token to a few, the pool nearly empty
        _case("plan-777-tight", "plan", streams=777, layout=3, page=32,
              frame_h=9, frame_w=11, chunk=99, new_lo=1, new_hi=40, kv_lo=1,
              kv_hi=4000, idle=11, tight=True, spare=63),
        # a single token of one stream: the launch is what counts
        _case("write-1", "write", kv_lo=7801, kv_hi=7801, chunk=1),
        # the 480p chunk of the 12-head model
        _case("write-480p-h12", "write", new_lo=4680, new_hi=4680,
              kv_lo=4680, kv_hi=4680, whole=True, spare=3),
        # four 720p chunks of the 40-head model in one step
        _case("write-720p-4x-h40", "write", streams=4, layout=4, heads=40,
              kv_heads=40, page=128, frame_h=45, frame_w=80, chunk=10800,
              new_lo=10800, new_hi=10800, kv_lo=3600, kv_hi=10800),
        # one token over the short 480p cache: latency and 48 MB of cache
        _case("attn-1tok-h12", "attn", kv_lo=7799, kv_hi=7799, chunk=1),
        # single tokens of 24 streams, grouped heads, ragged caches, pages
        # of 16 tokens
        _case("attn-24tok-gqa", "attn", streams=24, layout=5, heads=40,
              kv_heads=8, page=16, kv_lo=100, kv_hi=32760, chunk=1),
        # parts of frames: 20 to 400 rows of six streams
        _case("attn-part-h12", "attn", streams=6, layout=6, new_lo=20,
              new_hi=400, kv_lo=1560, kv_hi=32760, page=32, spare=11),
        # the 480p chunk over the cache of an 81-frame video, 12 heads
        _case("attn-480p-h12", "attn", new_lo=4680, new_hi=4680,
              kv_lo=28080, kv_hi=28080, whole=True),
        # five streams of the 12-head model, a long one past its window
        _case("attn-5x-capped", "attn", streams=5, layout=7, page=16,
              new_lo=1560, new_hi=4680, kv_lo=15600, kv_hi=93600,
              window=65520, chunk=4680, spare=77),
        # the last chunk of a 165-frame video of the 40-head model
        _case("attn-480p-165f-h40", "attn", heads=40, kv_heads=40,
              new_lo=4680, new_hi=4680, kv_lo=60840, kv_hi=60840,
              whole=True),
    ]


def _logint(rng, lo, hi):
    if hi <= lo:
        return lo
    if lo > 0 and hi > 10 * lo:
        return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo),
                                                        math.log(hi + 1))))))
    return rng.randint(lo, hi)


def draw(rng):
    op = rng.choice(("plan", "write", "attn", "attn"))
    heads, kv_heads = rng.choice(((2, 2), (12, 12), (40, 40), (40, 8),
                                  (16, 2), (7, 7), (8, 1), (12, 4)))
    page = rng.choice((16, 32, 64, 128))
    fh, fw = rng.choice(((30, 52), (45, 80), (9, 11), (16, 16), (23, 40)))
    frames = rng.choice((1, 2, 3))
    c = _case(None, op, layout=rng.randint(10, 10 ** 6), heads=heads,
              kv_heads=kv_heads, page=page, frame_h=fh, frame_w=fw,
              chunk=frames * fh * fw, spare=rng.choice((0, 0, 1, 50, 300)))
    del c["name"]
    longest = 900 * fh * fw          # positions stay inside the RoPE grid
    if op == "plan":
        c["streams"] = _logint(rng, 1, 1000)
        c["new_lo"] = 1
        c["new_hi"] = min(_logint(rng, 1, 5000), 150000 // c["streams"] + 1)
        c["kv_hi"] = min(longest, 60000, 1500000 // c["streams"])
        c["window"] = rng.choice((0, 0, c["chunk"] * rng.randint(1, 8)))
        c["ended"] = rng.choice((0, 3, 10))
        c["idle"] = rng.choice((0, 4, 9))
        c["tight"] = rng.random() < 0.3
    elif op == "write":
        c["streams"] = _logint(rng, 1, 40)
        c["new_hi"] = min(_logint(rng, 1, 10800),
                          1 + 40000 * 12 // (c["streams"] * heads))
        c["new_lo"] = max(1, c["new_hi"] // 3)
        c["kv_hi"] = min(longest, 4000)
        c["idle"] = rng.choice((0, 4))
    else:
        few = rng.random() < 0.45
        c["streams"] = _logint(rng, 1, 40 if few else 6)
        if few:
            c["new_hi"] = max(1, rng.choice((1, 1, 2, 4, 16)) * kv_heads
                              // heads)
            c["chunk"] = rng.choice((1, 1, 16, c["chunk"]))
        else:
            c["new_hi"] = _logint(rng, 17, 4680)
        c["new_lo"] = max(1, c["new_hi"] // 2)
        c["kv_hi"] = min(longest, _logint(rng, 300, 65000),
                         2000000 // c["streams"])
        c["kv_lo"] = rng.choice((0, c["kv_hi"] // 2, c["kv_hi"]))
        c["window"] = rng.choice((0, 0, 0, c["chunk"] * rng.randint(1, 20),
                                  5000))
        c["idle"] = rng.choice((0, 0, 3))
        while work(c)["flops"] > 4e12:
            c["new_hi"] = max(1, c["new_hi"] // 2)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
    return c


class _Stream:
    """Lengths of one stream before a step; new < 0 ends it."""

    def __init__(self, old, new, first):
        self.old, self.new, self.first = old, new, first


def _lo(case, a):
    """First position that the query at position a sees."""
    if case["window"] == 0:
        return 0
    return max(0, (a // case["chunk"] + 1) * case["chunk"] - case["window"])


def _hi(case, a, kv):
    return min(kv, (a // case["chunk"] + 1) * case["chunk"])


def _layout(case):
    """The streams' lengths, from the case alone."""
    rng = random.Random(case["layout"])
    out = []
    for r in range(case["streams"]):
        old = _logint(rng, case["kv_lo"], case["kv_hi"])
        if case["whole"]:
            old -= old % case["chunk"]
        new = _logint(rng, case["new_lo"], case["new_hi"])
        if case["idle"] and r % case["idle"] == case["idle"] - 1:
            new = 0
        if case["ended"] and r % case["ended"] == case["ended"] - 1:
            new = -1
        # pages the stream's previous step already gave back
        prev = max(0, old - max(1, min(case["chunk"], case["new_hi"])))
        first = min(_lo(case, prev), prev) // case["page"]
        out.append(_Stream(old, new, first))
    return out


def _up(a, b):
    return -(-a // b)


def _sizes(case):
    """(streams, max_pages, n_pages, token_cap, RoPE frames)."""
    ps = case["page"]
    st = _layout(case)
    hw = case["frame_h"] * case["frame_w"]
    last = max(s.old + max(s.new, 0) for s in st)
    held = sum(_up(s.old, ps) - s.first for s in st)
    need = sum(_up(s.old + max(s.new, 0), ps) - _up(s.old, ps) for s in st)
    ends = sum(_up(s.old, ps) - s.first for s in st if s.new < 0)
    n_pages = held + 3 + (max(0, need * 3 // 4 - ends) if case["tight"]
                          else need + need // 8)
    cap = sum(max(s.new, 0) for s in st) + case["spare"]
    return st, _up(last, ps) + 2, n_pages, max(cap, 1), _up(max(last, 1), hw)


def work(case):
    st, max_pages, n_pages, cap, frames = _sizes(case)
    ps, R = case["page"], case["streams"]
    T = sum(max(s.new, 0) for s in st)
    h, kvh = case["heads"], case["kv_heads"]
    if case["op"] == "plan":
        moved = 0
        for s in st:
            if s.new < 0:
                moved += _up(s.old, ps) - s.first
            elif s.new > 0:
                moved += max(0, min(_lo(case, s.old), s.old) // ps - s.first)
                moved += _up(s.old + s.new, ps) - _up(s.old, ps)
        # lengths and settings in, lengths and status out, each moved page
        # read from one list, written to another and its old entry cleared,
        # one record a token
        return {"bytes": R * (4 + 16 + 8 + 8 + 12) + 12 * moved + 16 * cap,
                "flops": 0}
    if case["op"] == "write":
        return {"bytes": 2 * T * (h + 2 * kvh) * HD * 2 + 16 * cap
                + (h + kvh) * HD * 4,
                "flops": T * (h + kvh) * HD * 8}
    pairs = keys = 0
    for s in st:
        if s.new <= 0:
            continue
        kv = s.old + s.new
        a = s.old
        while a < kv:           # rows of one chunk see the same keys
            n = min(kv, (a // case["chunk"] + 1) * case["chunk"]) - a
            pairs += n * max(0, _hi(case, a, kv) - _lo(case, a))
            a += n
        keys += max(0, kv - _lo(case, s.old))
    return {"bytes": 2 * T * h * HD * 2 + 2 * keys * kvh * HD * 2,
            "flops": 4 * HD * h * pairs}


# ------------------------------------------------------------ preparation --

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _state(case, seed):
    """The cache's state before the step: lengths, block table, free pages."""
    st, max_pages, n_pages, cap, frames = _sizes(case)
    R, ps = case["streams"], case["page"]
    rng = random.Random(seed * 7919 + case["layout"])
    pages = list(range(n_pages))
    rng.shuffle(pages)
    table = torch.full((R, max_pages), -1, dtype=torch.int32)
    n = 0
    for r, s in enumerate(st):
        held = _up(s.old, ps) - s.first
        table[r, s.first:s.first + held] = torch.tensor(
            pages[n:n + held], dtype=torch.int32)
        n += held
    head = rng.randrange(n_pages)
    ring = [-1] * n_pages
    for i, p in enumerate(pages[n:]):
        ring[(head + i) % n_pages] = p
    cfg = [[case["frame_h"], case["frame_w"], case["chunk"], case["window"]]]
    return dict(streams=_i32(cfg * R), kv_lens=_i32([s.old for s in st]),
                first_pages=_i32([s.first for s in st]),
                block_table=table.to(DEV), free_ring=_i32(ring),
                ring_state=_i32([head, n_pages - n]),
                new_lens=_i32([s.new for s in st]))


def _randn(shape, gen, scale=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):     # fp32 draws, by parts
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device=DEV) * scale
    return out


def _cos_sin(frames, fh, fw):
    """cos and sin of every position of the three axes, fp32."""
    out = []
    for n, width in ((frames, 44), (fh, 42), (fw, 42)):
        freq = THETA ** (-2.0 * torch.arange(width // 2, dtype=torch.float64)
                         / width)
        ang = torch.arange(n, dtype=torch.float64)[:, None] * freq
        out.append((ang.cos().float().to(DEV), ang.sin().float().to(DEV)))
    return out


def _inputs(case, seed):
    """Everything drawn from the seed."""
    st, max_pages, n_pages, cap, frames = _sizes(case)
    h, kvh = case["heads"], case["kv_heads"]
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003
                                                  + case["layout"])
    state = dict(case=case, host=st, before=_state(case, seed),
                 grid=(frames, case["frame_h"], case["frame_w"]),
                 dims=(max_pages, n_pages, cap))
    if case["op"] == "plan":
        return state
    pool = (n_pages, kvh, case["page"], HD)
    state["q"] = _randn((cap, h, HD), gen)
    state["k_pages"] = _randn(pool, gen)
    state["v_pages"] = _randn(pool, gen)
    state["out"] = torch.zeros((cap, h, HD), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "write":
        state["k"] = _randn((cap, kvh, HD), gen, 2.0)
        state["v"] = _randn((cap, kvh, HD), gen)
        state["wq"] = torch.rand(h * HD, generator=gen, device=DEV) + 0.5
        state["wk"] = torch.rand(kvh * HD, generator=gen, device=DEV) + 0.5
    return state


def prepare(case, seed):
    state = _inputs(case, seed)
    s, (max_pages, n_pages, cap) = state["before"], state["dims"]
    if own:
        from video_diffusion_transformer_self_b200 import paged, wan
        g = wan.grid(*state["grid"])
        cache = paged.PagedCache(
            s["streams"], g, n_pages=n_pages, page_size=case["page"],
            max_pages=max_pages, heads=case["heads"],
            kv_heads=case["kv_heads"], token_cap=cap,
            max_new=max(1, max(x.new for x in state["host"])))
        for name in ("kv_lens", "first_pages", "block_table", "free_ring",
                     "ring_state"):
            getattr(cache, name).copy_(s[name])
        state.update(cache=cache, saved=cache.state.clone())
    if case["op"] == "plan":
        return state
    # the step's plan is made once, all layers and passes use it
    if own:
        cache.plan(s["new_lens"])
        state["rope"] = wan.rope3d_table(g, theta=THETA)
    else:
        planned = _plan(state)
        state.update(table=planned[2], tokens=planned[8],
                     rope=_cos_sin(*state["grid"]))
    return state


# ------------------------------------------------------------ plain forms --

def _plan(state):
    """The step's plan with elementary operations on whole arrays."""
    case, s = state["case"], state["before"]
    max_pages, n_pages, cap = state["dims"]
    F, gh, gw = state["grid"]
    ps = case["page"]
    i64 = torch.int64
    H, W, chunk, window = (c.to(i64) for c in s["streams"].unbind(1))
    old, first = s["kv_lens"].to(i64), s["first_pages"].to(i64)
    new = s["new_lens"].to(i64)
    table = s["block_table"].to(i64)
    ring = s["free_ring"].to(i64)
    head, count = s["ring_state"].to(i64).unbind(0)
    ended = new < 0
    rows = new.clamp(min=0)
    end = rows.cumsum(0)
    start = end - rows
    total = old + rows
    fit = ((H >= 1) & (W >= 1) & (H <= gh) & (W <= gw) & (chunk >= 1)
           & (window >= 0) & (total <= max_pages * ps)
           & (total <= F * H * W) & (end <= cap))
    valid = (new > 0) & fit
    # pages that go back to the ring
    held = (old + ps - 1) // ps
    lo = ((old // chunk.clamp(min=1) + 1) * chunk - window).clamp(min=0)
    lo = torch.where(window > 0, lo, torch.zeros_like(lo))
    gone = torch.maximum(first, torch.minimum(lo, old) // ps)
    gone = torch.where(valid, gone, first)
    gone = torch.where(ended, held, gone)
    freed = gone - first
    at = freed.cumsum(0) - freed
    col = torch.arange(max_pages, device=DEV)[None]
    back = (col >= first[:, None]) & (col < gone[:, None])
    dest = (head + count + at[:, None] + col - first[:, None]) % n_pages
    # entries that do not go back aim at one slot past the ring
    dest = torch.where(back, dest, torch.full_like(dest, n_pages))
    ring = torch.cat([ring, ring.new_zeros(1)])
    ring.scatter_(0, dest.view(-1), table.view(-1))
    ring = ring[:n_pages]
    table = torch.where(back, torch.full_like(table, -1), table)
    count = count + freed.sum()
    # pages for the new tokens, in the streams' order
    top = (total + ps - 1) // ps
    need = torch.where(valid, top - held, torch.zeros_like(top))
    upto = need.cumsum(0)
    room = upto <= count
    admit = valid & room
    src = (head + (upto - need)[:, None] + col - held[:, None]) % n_pages
    take = admit[:, None] & (col >= held[:, None]) & (col < top[:, None])
    table = torch.where(take, ring[src], table)
    used = torch.where(admit, need, torch.zeros_like(need)).sum()
    q_lens = torch.where(admit, new, torch.zeros_like(new))
    status = torch.where((new > 0) & ~fit, -1, torch.where(valid & ~room, -6,
                                                          0))
    kv = torch.where(ended, torch.zeros_like(old), old + q_lens)
    first = torch.where(ended, torch.zeros_like(first), gone)
    # one record a packed row: time, height, width, slot
    i = torch.arange(cap, device=DEV)
    r = torch.searchsorted(end, i, right=True).clamp(max=len(end) - 1)
    off = i - start[r]
    live = (off >= 0) & (off < q_lens[r])
    a = old[r] + off
    hw = (H * W).clamp(min=1)[r]
    page = table[r, (a // ps).clamp(max=max_pages - 1)]
    rec = torch.stack([a // hw, a % hw // W.clamp(min=1)[r],
                       a % W.clamp(min=1)[r], page * ps + a % ps], 1)
    none = torch.tensor([0, 0, 0, -1], device=DEV)
    rec = torch.where(live[:, None], rec, none)
    q_start = torch.cat([start.clamp(max=cap), end[-1:].clamp(max=cap)])
    ring_state = torch.stack([(head + used) % n_pages, count - used])
    return [x.to(torch.int32) for x in (kv, first, table, ring, ring_state,
                                        q_start, q_lens, status, rec)]


def _norm_rope(x, w, pos, rope):
    x = x.float()
    f = torch.rsqrt(x.square().mean((1, 2), keepdim=True) + EPS)
    x = x * f * w.view(1, -1, HD)
    c = torch.cat([rope[i][0][pos[:, i]] for i in range(3)], 1)[:, None]
    s = torch.cat([rope[i][1][pos[:, i]] for i in range(3)], 1)[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _write(state):
    ps = state["case"]["page"]
    n = sum(max(s.new, 0) for s in state["host"])     # rows of streams
    rec = state["tokens"][:n].long()
    out, kp, vp = state["out"], state["k_pages"], state["v_pages"]
    out[:n] = _norm_rope(state["q"][:n], state["wq"], rec,
                         state["rope"]).to(out.dtype)
    page, off = rec[:, 3] // ps, rec[:, 3] % ps
    kp[page, :, off] = _norm_rope(state["k"][:n], state["wk"], rec,
                                  state["rope"]).to(kp.dtype)
    vp[page, :, off] = state["v"][:n]
    return [out, kp, vp]


def _attn(state):
    case = state["case"]
    ps, h, kvh = case["page"], case["heads"], case["kv_heads"]
    group = h // kvh
    scale = 1.0 / math.sqrt(HD)
    out = state["out"]
    row = 0
    for r, s in enumerate(state["host"]):
        n = max(s.new, 0)
        if n == 0:
            continue
        kv = s.old + n
        p0 = min(_lo(case, s.old), kv - 1) // ps
        j = torch.arange(p0 * ps, kv, device=DEV)
        ids = state["table"][r, p0:_up(kv, ps)].long()
        # heads by parts, so that the scores stay under about 2 GB
        step = max(1, min(kvh, (1 << 29) // (group * n * len(j))))
        a = torch.arange(s.old, kv, device=DEV)
        hi = (a // case["chunk"] + 1) * case["chunk"]
        lo = hi - case["window"] if case["window"] else torch.zeros_like(hi)
        hide = (j[None] >= hi[:, None]) | (j[None] < lo[:, None])
        for h0 in range(0, kvh, step):
            h1 = min(kvh, h0 + step)
            k = state["k_pages"][ids, h0:h1].float().transpose(0, 1)
            v = state["v_pages"][ids, h0:h1].float().transpose(0, 1)
            k = k.reshape(h1 - h0, -1, HD)[:, :len(j)]
            v = v.reshape(h1 - h0, -1, HD)[:, :len(j)]
            q = state["q"][row:row + n, h0 * group:h1 * group].float()
            q = q.view(n, h1 - h0, group, HD).permute(1, 2, 0, 3)
            x = q.reshape(h1 - h0, group * n, HD) @ k.transpose(1, 2)
            x = x.view(h1 - h0, group, n, len(j)).mul_(scale)
            x.masked_fill_(hide, -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            x = x.sub_(m).exp_()
            t = x.sum(-1, keepdim=True)
            o = x.view(h1 - h0, group * n, len(j)) @ v
            o = o.view(h1 - h0, group, n, HD) / torch.where(
                t == 0, torch.ones_like(t), t)
            out[row:row + n, h0 * group:h1 * group] = o.permute(
                2, 0, 1, 3).reshape(n, -1, HD).to(out.dtype)
        row += n
    return [out]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"plan": _plan, "write": _write, "attn": _attn}[op](state)
    cache = state["cache"]
    if op == "plan":
        # the same step again: the state as it was before it
        cache.state.copy_(state["saved"])
        cache.plan(state["before"]["new_lens"])
        return [cache.kv_lens, cache.first_pages, cache.block_table,
                cache.free_ring, cache.ring_state, cache.q_start,
                cache.q_lens, cache.status, cache.tokens]
    if op == "write":
        cache.write(state["q"], state["k"], state["v"], state["wq"],
                    state["wk"], state["rope"], state["k_pages"],
                    state["v_pages"], q_out=state["out"], eps=EPS)
        return [state["out"], state["k_pages"], state["v_pages"]]
    cache.attn(state["q"], state["k_pages"], state["v_pages"], state["out"])
    return [state["out"]]


# ------------------------------------------------------------------ exact --

def _exact_plan(case, seed):
    """One stream after another, on the host."""
    st, max_pages, n_pages, cap, frames = _sizes(case)
    b = {k: v.cpu().tolist() for k, v in _state(case, seed).items()}
    ps, fh, fw = case["page"], case["frame_h"], case["frame_w"]
    kv, first, table = b["kv_lens"], b["first_pages"], b["block_table"]
    ring, (head, count) = b["free_ring"], b["ring_state"]
    R = len(kv)
    starts, at = [], 0
    for n in b["new_lens"]:
        starts.append(at)
        at += max(n, 0)
    fits = [at2 + max(n, 0) <= cap and kv[r] + max(n, 0) <= max_pages * ps
            and kv[r] + max(n, 0) <= frames * fh * fw
            for r, (n, at2) in enumerate(zip(b["new_lens"], starts))]
    for r, n in enumerate(b["new_lens"]):      # pages come back first
        upto = first[r]
        if n < 0:
            upto = _up(kv[r], ps)
        elif n > 0 and fits[r]:
            upto = max(upto, min(_lo(case, kv[r]), kv[r]) // ps)
        for p in range(first[r], upto):
            ring[(head + count) % n_pages] = table[r][p]
            table[r][p] = -1
            count += 1
        first[r] = upto
        if n < 0:
            kv[r] = first[r] = 0
    lens, status, rec = [0] * R, [0] * R, [[0, 0, 0, -1]] * cap
    stopped, used, q_start = False, 0, []
    for r, n in enumerate(b["new_lens"]):
        q_start.append(min(starts[r], cap))
        if n <= 0:
            continue
        if not fits[r]:
            status[r] = -1
            continue
        need = _up(kv[r] + n, ps) - _up(kv[r], ps)
        used += need
        stopped = stopped or used > count
        if stopped:
            status[r] = -6
            continue
        for p in range(_up(kv[r], ps), _up(kv[r] + n, ps)):
            table[r][p] = ring[(head + used - need) % n_pages]
            need -= 1
        for i in range(n):
            a = kv[r] + i
            t, rest = divmod(a, fh * fw)
            rec[starts[r] + i] = [t, rest // fw, rest % fw,
                                  table[r][a // ps] * ps + a % ps]
        kv[r] += n
        lens[r] = n
    took = sum(_up(kv[r], ps) - _up(kv[r] - lens[r], ps) for r in range(R))
    return [_i32(x) for x in (kv, first, table, ring,
                              [(head + took) % n_pages, count - took],
                              q_start + [min(at, cap)], lens, status, rec)]


def _exact_write(case, seed):
    state = _inputs(case, seed)
    planned = _exact_plan(case, seed)
    ps = case["page"]
    rec = planned[8].long()
    live = (rec[:, 3] >= 0).nonzero()[:, 0]
    rec = rec[live]
    ang = []
    for axis, width in ((0, 44), (1, 42), (2, 42)):
        e = torch.arange(0, width, 2, dtype=torch.float64, device=DEV) / width
        ang.append(rec[:, axis].double()[:, None] * torch.pow(
            torch.tensor(THETA, dtype=torch.float64, device=DEV), -e))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.cat(ang, 1))
    out = state["out"].double()
    kp, vp = state["k_pages"].double(), state["v_pages"].double()

    def turned(x, w):
        x = x[live].double()
        ms = x.flatten(1).pow(2).sum(1) / (x.shape[1] * HD)
        x = x / torch.sqrt(ms + EPS)[:, None, None]
        x = x * w.double().view(-1, HD)
        z = torch.view_as_complex(x.unflatten(-1, (64, 2))) * turn[:, None]
        return torch.view_as_real(z).flatten(-2)

    out[live] = turned(state["q"], state["wq"])
    page = torch.div(rec[:, 3], ps, rounding_mode="floor")
    kp[page, :, rec[:, 3] - page * ps] = turned(state["k"], state["wk"])
    vp[page, :, rec[:, 3] - page * ps] = state["v"][live].double()
    return [out, kp, vp]


def _exact_attn(case, seed):
    state = _inputs(case, seed)
    table = _exact_plan(case, seed)[2].long()
    ps, h, kvh = case["page"], case["heads"], case["kv_heads"]
    out = state["out"].double()
    row = 0
    for r, s in enumerate(_layout(case)):
        n = max(s.new, 0)
        kv = s.old + n
        a0 = 0
        while a0 < n:           # rows that see the same keys
            a = s.old + a0
            upto = (a // case["chunk"] + 1) * case["chunk"]
            lo, hi = _lo(case, a), min(kv, upto)
            rows = min(kv, upto) - a
            rows = min(rows, max(1, (1 << 27) // max(1, hi - lo)))
            j = torch.arange(lo, max(lo, hi), device=DEV)
            for head in range(h):
                if len(j) == 0:
                    continue
                g = head // (h // kvh)
                k = state["k_pages"][table[r, j // ps], g, j % ps].double()
                v = state["v_pages"][table[r, j // ps], g, j % ps].double()
                at = slice(row + a0, row + a0 + rows)
                x = (state["q"][at, head].double() @ k.T) * HD ** -0.5
                out[at, head] = torch.exp(
                    x - torch.logsumexp(x, 1, keepdim=True)) @ v
            a0 += rows
        row += n
    return [out]


def exact(case, seed):
    if case["op"] == "plan":
        return _exact_plan(case, seed)
    if case["op"] == "write":
        return _exact_write(case, seed)
    # token-causal rows are taken one by one: long ones would take too long
    if case["chunk"] < 64 and case["streams"] * case["new_hi"] \
            * case["heads"] > 20000:
        return None
    return _exact_attn(case, seed)
