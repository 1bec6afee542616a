"""Gradients whose sink tiles are cut into pieces: the workspace's size, what
is written into it, and the sums."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api, build
from test_gpu_attn_ragged import _compare


def need(Tq, Hq, Hkv, D, B, max_q, window, sinks, Tk=None, max_k=None):
    build.build()
    return api.lib().bl_attn_backward_workspace_bytes(Tq, Tk or Tq, Hq, Hkv, D, B, max_q, max_k or max_q, window, sinks)


@pytest.mark.parametrize("Tq,Hq,Hkv,D,B,max_q,window,sinks", [
    (20000, 20, 20, 128, 16, 8192, 128, 4),
    (40000, 20, 20, 128, 32, 32768, 100, 4),          # one long entry among short ones
    (32768, 8, 8, 128, 1, 32768, 100, 1 << 40),       # every key a sink
    (32768, 8, 8, 128, 1, 32768, 100, 16000),
    (65536, 12, 4, 64, 65535, 500, 1, 1),
    (1 << 24, 1, 1, 16, 1, (1 << 24) - 1, 1, 1 << 23),
])
def test_workspace_grows_with_the_tokens(Tq, Hq, Hkv, D, B, max_q, window, sinks):
    """Tq * Hq floats (rounded up to 256 bytes) and at most 4 * Tq * Hkv * D more, whatever B * max_q is."""
    n = need(Tq, Hq, Hkv, D, B, max_q, window, sinks)
    assert 4 * Tq * Hq <= n <= 4 * Tq * Hq + 256 + 16 * Tq * Hkv * D


def test_workspace_without_pieces():
    for window, sinks, max_q in ((0, 4, 5000), (100, 0, 5000), (5000, 4, 5000), (100, 4, 512)):
        assert need(5000, 2, 1, 64, 10, max_q, window, sinks) == 40192


CASES = [
    # queries, keys, Hq, Hkv, D, window, sinks
    ([1100, 30, 1025], [1100, 30, 1025], 2, 1, 64, 100, 3),          # two cut entries, a short one between
    ([1200], [1200], 2, 2, 128, 60, 200),                            # sinks in two tiles
    ([5, 900, 900], [5, 900, 900], 2, 1, 96, 128, 129),
    ([640, 1290], [900, 1400], 2, 1, 64, 1, 127),                    # keys before the first query
    ([1300], [1200], 1, 1, 32, 30, 128),                             # queries that see nothing
    ([1500], [1500], 1, 1, 64, 200, 900),                            # most keys are sinks: not cut
]


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,window,sinks", CASES)
def test_gradients(nq, nk, Hq, Hkv, D, window, sinks):
    """With a workspace of exactly the size asked for, full of NaN, and what lies behind it untouched."""
    g = torch.Generator().manual_seed(sum(nq) + sinks)
    q, do = (torch.randn(sum(nq), Hq, D, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(sum(nk), Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    cu = [torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda() for n in (nq, nk)]
    most = (max(nq), max(nk))
    o, lse = api.bl_attn_forward(q, k, v, *cu, *most, window, sinks)
    size = need(sum(nq), Hq, Hkv, D, len(nq), most[0], window, sinks, sum(nk), most[1])
    buf = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    grads = api.bl_attn_backward(do, q, k, v, o, lse, *cu, *most, window, sinks, workspace=buf[:size])
    api.bl_check_device_error()
    assert bool((buf[size:] == 0xff).all())
    _compare(nq, nk, Hq, Hkv, D, window, sinks, D ** -0.5, q, k, v, do, o, lse, grads)
    again = api.bl_attn_backward(do, q, k, v, o, lse, *cu, *most, window, sinks)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
