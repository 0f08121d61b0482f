"""Key ranges of the block-causal kernels where some rows of a warp see no key
of a range while the maximum of others moves by more than 2^8 in it."""

import numpy as np
import pytest
import torch

from gpu_common import cuda, f64, scale_for
from oracle import attention as oattn
from paged_common import assert_attn
from video_diffusion_transformer_self_b200 import build, inputs, wan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wan.lib()


@pytest.mark.parametrize("pair", [False, True], ids=["tiles", "pair"])
@pytest.mark.parametrize("chunk,n_split", [(1000, 2), (1000, 4), (900, 3)])
def test_rows_without_keys_beside_rows_whose_maximum_moves(chunk, n_split,
                                                           pair):
    L = 2 * chunk
    q = inputs.randn_bf16((1, L, 2, 128), 70 + n_split, 8.0)
    k = inputs.randn_bf16((1, L, 2, 128), 71 + n_split)
    v = inputs.randn_bf16((1, L, 2, 128), 72 + n_split)
    o = torch.empty_like(cuda(q))
    wan.block_causal_attn(cuda(q), cuda(k), cuda(v), o, chunk, pair=pair,
                          split=n_split)
    torch.cuda.synchronize()
    assert wan.device_status() == 0
    # the roundings of the attention over pages are those of these kernels
    want, mag = (oattn.block_causal_attention(f64(q), f64(k), x, scale_for(),
                                              chunk)
                 for x in (f64(v), np.abs(f64(v))))
    score_sum = scale_for() * float(q.float().norm(dim=-1).max()
                                    * k.float().norm(dim=-1).max())
    assert_attn(f64(o), want, mag, "chunk %d, %d ranges" % (chunk, n_split),
                score_sum)


def test_scratch_of_a_call_on_another_stream_is_not_handed_out_meanwhile():
    L, chunk, n_split = 2048, 1024, 2
    q, k, v = (cuda(inputs.randn_bf16((1, L, 2, 128), 90 + i))
               for i in range(3))
    o = torch.empty_like(q)
    want = torch.empty_like(q)
    wan.block_causal_attn(q, k, v, want, chunk, split=n_split)
    need = wan.block_causal_workspace_bytes(1, L, 2, n_split)
    side = torch.cuda.Stream()
    # (the fill kernel is loaded now: loading waits for the device)
    assert bool((torch.full((need,), 77, dtype=torch.uint8,
                            device="cuda") == 77).all())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)      # some 50 ms before the kernels
    wan.block_causal_attn(q, k, v, o, chunk, split=n_split, stream=side)
    later = torch.full((need,), 77, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((later == 77).all())
    assert torch.equal(o, want)
