"""The place -> unit arithmetic that the plan cuts the attention's work with
and the attention walks it with (csrc/paged.cuh), compiled for the host and
compared with Python integers, up to the largest sizes a cache may have."""

import ctypes
import os
import random
import subprocess

import pytest

from video_diffusion_transformer_self_b200 import build, wan

CSRC = os.path.join(build.PKG, "csrc")
SOURCE = r"""
#include "paged.cuh"
extern "C" int unit_of(int64_t y, int tiles, int full, int last, int* tile,
                       int* weight, int* off) {
  return wan::paged::unit_of(y, tiles, full, last, tile, weight, off);
}
extern "C" int64_t weight_before(int n, int tiles, int full, int last) {
  return wan::paged::weight_before(n, tiles, full, last);
}
extern "C" int work_kind(const wan_paged_t* c) {
  return wan::paged::work_kind(c);
}
extern "C" int pair_weight(int nb) {
  return wan::paged::kPairWeight * nb + wan::paged::kUnitWeight;
}
extern "C" int one_weight(int nb) {
  return wan::paged::kOneWeight * nb + wan::paged::kUnitWeight;
}
"""


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, so = str(d / "units.cu"), str(d / "units.so")
    with open(src, "w", encoding="utf-8") as f:
        f.write(SOURCE)
    subprocess.run([build.NVCC] + build.FLAGS + ["-I", CSRC, src, "-o", so],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(so)
    lib.unit_of.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 3 \
        + [ctypes.POINTER(ctypes.c_int)] * 3
    lib.weight_before.restype = ctypes.c_int64
    return lib


# (head groups, new tokens, tokens of a tile pair, keys).  The first ones are
# ordinary chunks; from the fourth on a head group's units weigh 2^32 and more.
SIZES = [
    (12, 4680, 256, 32760), (40, 43200, 256, 65520), (1, 17, 256, 17),
    (1, 1048576, 16, 1048576), (1, 2097152, 16, 2097152),
    (1, 1500000, 32, 1500000), (1, 4194304, 256, 4194304),
    (1, 1200000, 16, 1200000), (1, 300000, 16, 4000000),
    (1, 1 << 27, 16, 1 << 30), (15, 1 << 27, 256, 1 << 30),
    (1023, 1 << 21, 256, 1 << 30), (1024, 1000, 256, 1 << 30)]


@pytest.mark.parametrize("groups,ql,pair,keys", SIZES)
def test_every_place_maps_to_its_unit(units, groups, ql, pair, keys):
    tiles = -(-ql // pair)
    nb = -(-keys // 128)
    while nb > 65535:           # as the plan scales its lengths
        nb >>= 1
    full = units.pair_weight(nb)
    rest = ql % pair
    rng = random.Random(ql + keys)
    for last in (full, units.one_weight(nb)):
        if last != full and not 1 <= rest <= pair // 2:
            continue
        n_units = groups * tiles
        picks = {0, 1, tiles - 1, tiles, n_units - 2, n_units - 1}
        picks.update(rng.randrange(n_units) for _ in range(400))
        t, w, o = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        for n in sorted(p for p in picks if 0 <= p < n_units):
            g, tile = divmod(n, tiles)
            size = full if tile else last
            start = g * ((tiles - 1) * full + last) \
                + (last + (tile - 1) * full if tile else 0)
            assert units.weight_before(n, tiles, full, last) == start
            for off in (0, 1, size // 2, size - 1):
                got = units.unit_of(start + off, tiles, full, last, t, w, o)
                assert (got, t.value, w.value, o.value) == \
                    (g, tile, size, off), (n, off)


def test_work_lists_of_other_layouts_have_other_kinds(units):
    def kind(heads, kv_heads, max_new):
        d = wan.PagedDesc()
        d.heads, d.kv_heads, d.max_new = heads, kv_heads, max_new
        return units.work_kind(ctypes.byref(d))

    # few rows: their number; tiles: the heads of a tile, which long steps of
    # groups like 5 and 7 do not share
    assert kind(8, 8, 16) != kind(8, 8, 17)
    assert kind(8, 8, 16) != kind(8, 8, 2)
    assert kind(5, 1, 1024) != kind(5, 1, 1025)
    assert kind(8, 8, 700) == kind(8, 8, 1 << 27)
    assert kind(8, 2, 1024) == kind(8, 2, 1025)
    seen = {}
    for heads in (1, 2, 7, 8, 40, 512, 1024):
        for kv_heads in range(1, heads + 1):
            if heads % kv_heads == 0:
                group = heads // kv_heads
                for rows in range(group, 17, group):
                    k = kind(heads, kv_heads, rows // group)
                    assert k > 0 and k not in seen
                    seen[k] = (heads, kv_heads, rows)
                k = kind(heads, kv_heads, 1 << 20)
                assert k > 0 and k not in seen
                seen[k] = (heads, kv_heads, 0)
