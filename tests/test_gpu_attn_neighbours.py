"""An entry of a ragged batch gives the same bits whatever is packed around it."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
@pytest.mark.parametrize("n", [300, 517])
def test_same_bits_alone_and_packed(n, window, sinks, D):
    """Entries of several key tiles whose last warp holds rows of the next one, whose scores are thirty times
    larger (their maxima move in tile after tile)."""
    g = torch.Generator().manual_seed(n + D)
    T, Hq, Hkv = 100 + n + 200, 4, 2
    q, do = (torch.randn(T, Hq, D, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    q[100 + n:] *= 30
    q[:100] *= 30
    cu = torch.tensor([0, 100, 100 + n, T], dtype=torch.int32).cuda()
    o, lse = api.bl_attn_forward(q, k, v, cu, cu, n, n, window, sinks)
    grads = api.bl_attn_backward(do, q, k, v, o, lse, cu, cu, n, n, window, sinks)
    rows = slice(100, 100 + n)
    alone = [t[rows].contiguous() for t in (do, q, k, v)]
    cu1 = torch.tensor([0, n], dtype=torch.int32).cuda()
    o1, lse1 = api.bl_attn_forward(*alone[1:], cu1, cu1, n, n, window, sinks)
    grads1 = api.bl_attn_backward(*alone, o1, lse1, cu1, cu1, n, n, window, sinks)
    api.bl_check_device_error()
    assert torch.equal(lse[:, rows], lse1) and torch.equal(o[rows], o1)
    assert all(torch.equal(a[rows], b) for a, b in zip(grads, grads1))
