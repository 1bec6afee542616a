"""Entries longer than max_q or max_k say: reported, and nothing that was not computed is read."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api

pytestmark = pytest.mark.gpu
INDEX = 9


def _reported():
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == INDEX


@pytest.mark.parametrize("D,Hkv", [(64, 2), (128, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0)])
def test_longer_than_declared(D, Hkv, window, sinks):
    n, some = 700, 100
    g = torch.Generator().manual_seed(D)
    q, do = (torch.randn(n, 2, D, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(n, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    o, lse = api.bl_attn_forward(q, k, v, cu, cu, n, n, window, sinks)
    head = do.clone()
    head[some:] = 0                              # rows that contribute exactly nothing
    want = api.bl_attn_backward(head, q, k, v, o, lse, cu, cu, n, n, window, sinks)
    full = api.bl_attn_backward(do, q, k, v, o, lse, cu, cu, n, n, window, sinks)
    api.bl_check_device_error()

    # queries: the gradients of the first `some`, whatever the workspace held before
    need = api.lib().bl_attn_backward_workspace_bytes(n, n, 2, Hkv, D, 1, some, n, window, sinks)
    for fill in (0x00, 0xff):
        work = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        dq = torch.full_like(q, 9.0)
        got = api.bl_attn_backward(do, q, k, v, o, lse, cu, cu, some, n, window, sinks, dq=dq, workspace=work)
        _reported()
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert torch.equal(dq[:some], want[0][:some]) and bool((dq[some:] == 9.0).all())
    o2, lse2 = torch.full_like(q, 9.0), torch.full_like(lse, 9.0)
    api.bl_attn_forward(q, k, v, cu, cu, some, n, window, sinks, o=o2, lse=lse2)
    _reported()
    assert bool((o2[some:] == 9.0).all()) and bool((lse2[:, some:] == 9.0).all())
    # (other rows of a warp may move its base: float32 sums, exp2 and lse's own rounding, on both sides)
    lim = 2 * ((n / 8 + 64) * 2.0 ** -23 + 2.0 ** -21 + 4 * 2.0 ** -24 * (lse.abs().max() + 1))
    assert bool((lse2[:, :some] - lse[:, :some]).abs().max() <= lim)

    # keys: the first `some` get their whole gradients, the others none
    dk, dv = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
    got = api.bl_attn_backward(do, q, k, v, o, lse, cu, cu, n, some, window, sinks, dk=dk, dv=dv)
    _reported()
    assert torch.equal(got[0], full[0])
    for a, b in ((dk, full[1]), (dv, full[2])):
        assert torch.equal(a[:some], b[:some]) and bool((a[some:] == 9.0).all())
