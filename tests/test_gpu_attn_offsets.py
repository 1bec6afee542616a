"""Gradients of ragged attention when keys and values have a mean (a bias of
their projections), against the formulas in 64 bits.

What is common to a row's dS then does not average out: an error e of delta =
rowsum(P o dP) moves dq by scale e sum_j P_j k_j.  The bounds therefore grant
delta no rounding of the forward's bfloat16 output.
"""
from __future__ import annotations

import math

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api
from _attention import EPS16, EPS32, attention, score_error, visible

pytestmark = pytest.mark.gpu

CASES = [
    # queries, keys, Hq, Hkv, D, window, sinks
    ([1000], [1000], 2, 1, 128, 0, 0),
    ([260, 1, 391], [260, 1, 391], 2, 2, 128, 20, 0),     # windows of few keys that straddle two tiles
    ([700], [700], 2, 1, 64, 100, 3),
    ([300, 129], [300, 129], 4, 2, 64, 0, 0),
    ([40, 200], [333, 420], 2, 1, 96, 0, 0),              # keys before the first query
    ([100], [100], 2, 2, 32, 0, 0),                       # one tile
    ([640], [640], 1, 1, 80, 300, 130),
]


@pytest.mark.parametrize("mean", [0.0, 2.0, 8.0])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,window,sinks", CASES)
def test_gradients(nq, nk, Hq, Hkv, D, window, sinks, mean):
    """Bounds.  The products' scores are the same bits in the forward and for dq,
    so the weights' sum is off 1 by `whole` only: the float32 sum, exp2 (2^-21)
    and the roundings of lse and of the scaled exponent.  A single weight is off
    by w, which scores' errors enter.  With x = dP - delta,
        dS' - dS = P (2 w (|x| + sum P |x|) + whole |delta| + errors of dP),
    and rounding to bfloat16 adds EPS16 |dS0|, dS0 = P (dP - delta0), and EPS16 P
    |delta0 - delta| where the difference to delta0 = rowsum(do o o) is put right;
    delta0 is off by the output's rounding, which so enters squared."""
    g = torch.Generator().manual_seed(sum(nq) + D)
    group, scale = Hq // Hkv, D ** -0.5
    q, do = (torch.randn(sum(nq), Hq, D, generator=g).bfloat16() for _ in range(2))
    k, v = ((torch.randn(sum(nk), Hkv, D, generator=g) + mean * torch.randn(Hkv, D, generator=g).sign()).bfloat16()
            for _ in range(2))
    cu = [torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda() for n in (nq, nk)]
    dev = [t.cuda() for t in (do, q, k, v)]
    o, lse = api.bl_attn_forward(*dev[1:], *cu, max(nq), max(nk), window, sinks)
    got = api.bl_attn_backward(*dev, o, lse, *cu, max(nq), max(nk), window, sinks)
    api.bl_check_device_error()
    q, k, v, do = (t.double() for t in (q, k, v, do))
    dk, dk_lim = torch.zeros_like(k), torch.zeros_like(k)
    a = b = 0
    for n, m in zip(nq, nk):
        see = visible(n, m, window, sinks)
        for h in range(Hq):
            qh, kh, vh, doh = q[a:a + n, h], k[b:b + m, h // group], v[b:b + m, h // group], do[a:a + n, h]
            ref, l, P = attention(qh, kh, vh, see, scale)
            d = torch.where(see, score_error(qh, kh, scale, D), 0.0).amax(1, keepdim=True)
            sums = (m / 8 + 64) * 2.0 ** -23
            top = torch.where(see, (scale * (qh @ kh.T)).abs(), 0.0).amax(1, keepdim=True)
            whole = sums + 2.0 ** -21 + 8 * EPS32 * (l.abs()[:, None] + top + 1)
            w = d + whole
            dP = doh @ vh.T
            delta = (P * dP).sum(1, keepdim=True)
            x = (dP - delta).abs()
            dp_err = (D + 4) * 2.0 ** -23 * (doh.abs() @ vh.abs().T)
            dp_err = dp_err + (P * dp_err).sum(1, keepdim=True) + sums * (P * dP.abs()).sum(1, keepdim=True)
            o_err = EPS16 * ref.abs() + 2 * (EPS16 + w) * (P @ vh.abs())
            off = (doh.abs() * o_err).sum(1, keepdim=True)
            real = P * (2 * w * (x + (P * x).sum(1, keepdim=True)) + whole * delta.abs() + dp_err)
            dS = P * (dP - delta)
            err = (real + EPS16 * dS.abs()) * (1 + EPS16)
            err_q = err + 2 * EPS16 * P * off
            dq = scale * dS @ kh
            lim = scale * (err_q + sums * (dS.abs() + P * off)) @ kh.abs()
            lim = lim + EPS16 * (dq.abs() + lim)
            e = (got[0][a:a + n, h].double().cpu() - dq).abs()
            assert bool((e <= lim).all()), ("dq", h, (e / lim).nan_to_num().max())
            rows = (n * group / 8 + 64) * 2.0 ** -23
            dk[b:b + m, h // group] += scale * dS.T @ qh
            dk_lim[b:b + m, h // group] += scale * (err + rows * dS.abs()).T @ qh.abs()
        a, b = a + n, b + m
    dk_lim = dk_lim + EPS16 * (dk.abs() + dk_lim)
    e = (got[1].double().cpu() - dk).abs()
    assert bool((e <= dk_lim).all()), ("dk", (e / dk_lim).nan_to_num().max())


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_one_key(D):
    """A row that sees one key has dS = 0: its dq is what rounding leaves, the square of a bfloat16 half step, not the step."""
    n, mean = 300, 8.0
    g = torch.Generator().manual_seed(D)
    q, do = (torch.randn(n, 1, D, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = ((torch.randn(n, 1, D, generator=g) + mean).bfloat16().cuda() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    o, lse = api.bl_attn_forward(q, k, v, cu, cu, n, n, 1)
    dq, dk, dv = api.bl_attn_backward(do, q, k, v, o, lse, cu, cu, n, n, 1)
    api.bl_check_device_error()
    c = lambda t: t[:, 0].double()  # noqa: E731
    dp = (c(do).abs() * c(v).abs()).sum(1)
    # delta0 - delta <= 2 EPS16 dp (o's rounding and P's); times EPS16 where it is rounded and put right; float32 sums of D
    # products, and exp2 and the exponent's roundings against scores of up to |s|
    s = (c(q) * c(k)).sum(1).abs() * D ** -0.5
    lim = (4 * EPS16 * EPS16 + 2 * (D + 4) * 2.0 ** -23 + 2.0 ** -20 + 8 * EPS32 * (s + 1)) * dp * D ** -0.5
    assert bool((c(dq).abs() <= lim[:, None] * c(k).abs() * (1 + EPS16)).all())
    assert math.isfinite(float(dv.double().abs().max()))
