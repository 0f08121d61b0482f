"""The paged calls refuse bad sizes and pointers before any device work (no
GPU needed): through the C ABI, and in the Python class's constructor."""

import ctypes

import pytest
import torch

from video_diffusion_transformer_self_b200 import build, paged, wan


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wan.lib()


def _desc(**kw):
    d = dict(n_streams=3, max_pages=8, n_pages=20, page_size=16,
             token_cap=64, max_new=64, heads=4, kv_heads=2)
    grid = kw.pop("grid", (4, 4, 4))
    ptr = {n: 4096 * (i + 1) for i, n in enumerate(
        ("streams", "kv_lens", "first_pages", "block_table", "free_ring",
         "ring_state", "q_start", "q_lens", "status", "tokens", "work"))}
    for k, v in kw.items():
        (ptr if k in ptr else d)[k] = v
    return wan.PagedDesc(*d.values(), wan.grid(*grid), *ptr.values())


P = [ctypes.c_void_p((1 << 20) + 4096 * i) for i in range(10)]
ODD = ctypes.c_void_p((1 << 20) + 8)


def _plan(lib, d):
    return lib.wan_paged_plan(d, P[0], None)


def _write(lib, d, **kw):
    a = dict(q=P[0], q_out=P[1], k=P[2], v=P[3], wq=P[4], wk=P[5], kp=P[6],
             vp=P[7], table=P[8], eps=1e-6)
    a.update(kw)
    return lib.wan_paged_write(d, *a.values(), None)


def _attn(lib, d, **kw):
    a = dict(q=P[0], kp=P[1], vp=P[2], o=P[3], scale=0.1, ws=P[4],
             n=1 << 40)
    a.update(kw)
    return lib.wan_paged_attn(d, *a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(n_streams=0), dict(n_streams=1025), dict(max_pages=0),
    dict(n_pages=0), dict(page_size=8), dict(page_size=48),
    dict(page_size=256), dict(token_cap=0), dict(max_new=0), dict(heads=0),
    dict(kv_heads=0), dict(heads=5), dict(heads=2048, kv_heads=2048),
    dict(grid=(0, 4, 4)), dict(grid=(4, 1025, 4)),
    dict(n_streams=1024, max_pages=1 << 21),        # table entries
    dict(max_pages=1 << 27),                        # positions of a stream
    dict(n_pages=1 << 29), dict(n_pages=(1 << 27) + 1, kv_heads=4),
    dict(token_cap=1 << 28), dict(streams=None), dict(kv_lens=None),
    dict(block_table=None), dict(tokens=None), dict(work=None)])
def test_bad_caches_are_refused_by_every_call(lib, bad):
    d = _desc(**bad)
    for call in (_plan, _write, _attn):
        assert call(lib, d) == wan.WAN_EINVAL


def test_misaligned_arrays(lib):
    for name in ("streams", "block_table", "tokens", "work"):
        d = _desc(**{name: 4096 + 4})
        for call in (_plan, _write, _attn):
            assert call(lib, d) == wan.WAN_EALIGN


def test_call_arguments(lib):
    d = _desc()
    assert lib.wan_paged_plan(None, P[0], None) == wan.WAN_EINVAL
    assert lib.wan_paged_plan(d, None, None) == wan.WAN_EINVAL
    for name in ("q", "q_out", "k", "v", "wq", "wk", "kp", "vp", "table"):
        assert _write(lib, d, **{name: None}) == wan.WAN_EINVAL
        assert _write(lib, d, **{name: ODD}) == wan.WAN_EALIGN
    for eps in (0.0, -1.0, float("nan")):
        assert _write(lib, d, eps=eps) == wan.WAN_EINVAL
    for kw in (dict(vp=P[6]), dict(k=P[0]), dict(q_out=P[2]),
               dict(q_out=P[3]), dict(q_out=P[6]), dict(q_out=P[7]),
               dict(k=P[6]), dict(v=P[7])):
        assert _write(lib, d, **kw) == wan.WAN_EINVAL
    for name in ("q", "kp", "vp", "o", "ws"):
        assert _attn(lib, d, **{name: None}) == wan.WAN_EINVAL
        assert _attn(lib, d, **{name: ODD}) == wan.WAN_EALIGN
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _attn(lib, d, scale=scale) == wan.WAN_EINVAL
    for other in (P[0], P[1], P[2]):
        assert _attn(lib, d, o=other) == wan.WAN_EINVAL


def test_sizes(lib):
    assert lib.wan_paged_work_bytes(0) == 0
    assert lib.wan_paged_work_bytes(1025) == 0
    assert lib.wan_paged_work_bytes(2) > lib.wan_paged_work_bytes(1) > 0
    assert lib.wan_paged_workspace_bytes(None) == 0


def test_cache_constructor_refuses():
    ok = dict(n_pages=4, page_size=16, max_pages=4, heads=2, token_cap=8)
    g = wan.grid(4, 4, 4)
    s = torch.ones(2, 4, dtype=torch.int32)
    for bad in (s.long(), s[:, :3], s.t(), s[0], torch.ones(0, 4).int(),
                torch.ones(1025, 4).int()):
        with pytest.raises(ValueError):
            paged.PagedCache(bad, g, **ok)
    for kw in (dict(page_size=24), dict(n_pages=0), dict(max_pages=0),
               dict(token_cap=0), dict(heads=3, kv_heads=2),
               dict(max_new=0), dict(heads=0)):
        with pytest.raises(ValueError):
            paged.PagedCache(s, g, **dict(ok, **kw))
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedCache(s, g, **ok)
