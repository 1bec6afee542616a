"""bl_attn_forward and bl_attn_backward against plain 64-bit attention and the
formulas of its gradients, entry by entry and head by head."""
from __future__ import annotations

import math

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api
from _attention import EPS16, EPS32, attention, score_error, visible

pytestmark = pytest.mark.gpu


def _inputs(nq, nk, Hq, Hkv, D, seed, behind=0, strided=False):
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(nq) + behind, sum(nk) + behind
    q, do = (torch.randn(Tq, Hq, D, generator=g).bfloat16() for _ in range(2))
    k, v = (torch.randn(Tk, Hkv, D, generator=g).bfloat16() for _ in range(2))
    for x, n in ((q, sum(nq)), (do, sum(nq)), (k, sum(nk)), (v, sum(nk))):
        x[n:] = float("nan")                      # rows behind the last entry belong to nobody
    if strided:
        qkv = torch.cat([q, k, v], 1).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = [torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda() for n in (nq, nk)]
    return q.cuda(), k.cuda(), v.cuda(), do.cuda(), cu


def _compare(nq, nk, Hq, Hkv, D, window, sinks, scale, q, k, v, do, o, lse, grads):
    """Bounds.  A score is off by d (score_error), a weight by d + 2^-21 and, where
    it enters a product, by half a bf16 step.  o adds its own rounding; delta
    = rowsum(do o o) then carries o's error, dS that and its own rounding.
    Sums in float32 add a rounding per partial sum (one per 8 terms and tile)."""
    group = Hq // Hkv
    c = lambda x: x.double().cpu()  # noqa: E731
    q, k, v, do = c(q), c(k), c(v), c(do)
    o, lse = c(o), lse.cpu().double()
    if grads is not None:
        grads = [c(x) for x in grads]
        dk_ref, dv_ref = torch.zeros_like(grads[1]), torch.zeros_like(grads[2])
        dk_lim, dv_lim = torch.zeros_like(grads[1]), torch.zeros_like(grads[2])
    a = b = 0
    for n, m in zip(nq, nk):
        see = visible(n, m, window, sinks)
        for h in range(Hq):
            qh, kh, vh, doh = q[a:a + n, h], k[b:b + m, h // group], v[b:b + m, h // group], do[a:a + n, h]
            ref, l, P = attention(qh, kh, vh, see, scale)
            empty = l == -math.inf
            d = torch.where(see, score_error(qh, kh, scale, D), 0.0)
            d = d.amax(1, keepdim=True) if m else torch.zeros(n, 1)
            sums = (m / 8 + 64) * 2.0 ** -23
            w = d + 2.0 ** -21 + sums                      # of a weight against its row's sum
            lim = (EPS16 + 2 * w) * (P @ vh.abs()) + EPS16 * (ref.abs() + (EPS16 + 2 * w) * (P @ vh.abs()))
            err = (o[a:a + n, h] - ref).abs()
            assert bool((err <= lim).all()), ("o", h, (err / lim).nan_to_num().max())
            got = lse[h, a:a + n]
            assert bool((got[empty] == -math.inf).all())
            assert bool(((got - l).abs()[~empty] <= (w[:, 0] + 4 * EPS32 * (l.abs() + 1))[~empty]).all())
            if grads is None:
                continue
            dP = doh @ vh.T
            delta = (doh * ref).sum(1, keepdim=True)
            dS = P * (dP - delta)
            dp_err = (D + 4) * 2.0 ** -23 * (doh.abs() @ vh.abs().T)
            delta_err = (doh.abs() * (lim + EPS32 * ref.abs())).sum(1, keepdim=True) + D * EPS32 * (doh * ref).abs().sum(1, keepdim=True)
            ds_err = P * (2 * w * (dP - delta).abs() + dp_err + delta_err) + EPS16 * dS.abs()
            ds_err = ds_err * (1 + EPS16)
            dq = scale * dS @ kh
            lim = scale * (ds_err + sums * dS.abs()) @ kh.abs()
            lim = lim + EPS16 * (dq.abs() + lim)
            err = (grads[0][a:a + n, h] - dq).abs()
            assert bool((err <= lim).all()), ("dq", h, (err / lim).nan_to_num().max())
            rows = (n * group / 8 + 64) * 2.0 ** -23
            dk_ref[b:b + m, h // group] += scale * dS.T @ qh
            dk_lim[b:b + m, h // group] += scale * (ds_err + rows * dS.abs()).T @ qh.abs()
            dv_ref[b:b + m, h // group] += P.T @ doh
            dv_lim[b:b + m, h // group] += ((EPS16 + 2 * w + rows) * P).T @ doh.abs()
        a, b = a + n, b + m
    if grads is not None:
        for name, got, ref, lim in (("dk", grads[1], dk_ref, dk_lim), ("dv", grads[2], dv_ref, dv_lim)):
            lim = lim + EPS16 * (ref.abs() + lim)
            err = (got - ref).abs()[:b]
            assert bool((err <= lim[:b]).all()), (name, (err / lim[:b]).nan_to_num().max())


CASES = [
    # queries, keys, Hq, Hkv, D, window, sinks
    ([1], [1], 1, 1, 64, 0, 0),
    ([5, 1, 130], [5, 1, 130], 2, 2, 128, 0, 0),
    ([300, 17], [300, 17], 6, 2, 64, 0, 0),
    ([257], [257], 3, 1, 128, 40, 3),
    ([129, 0, 64], [129, 0, 64], 4, 4, 80, 1, 0),
    ([500], [500], 2, 1, 64, 128, 130),        # sinks that end in the second tile
    ([700], [700], 2, 2, 32, 100, 1),          # a sink tile cut into pieces
    ([40, 3], [333, 200], 2, 1, 128, 0, 0),    # keys before the first query
    ([40, 130], [333, 260], 2, 1, 64, 50, 4),
    ([130, 20, 7], [100, 4, 0], 2, 2, 64, 0, 0),   # queries that see nothing, an entry without keys
    ([200], [150], 2, 1, 128, 30, 2),
    ([0, 90], [60, 90], 2, 1, 96, 20, 40),     # keys that nobody sees
    ([384], [384], 2, 1, 16, 0, 5),            # sinks without a window change nothing
    ([1100], [1100], 1, 1, 128, 16, 2),
]


@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,window,sinks", CASES)
def test_forward_and_gradients(nq, nk, Hq, Hkv, D, window, sinks):
    q, k, v, do, (cq, ck) = _inputs(nq, nk, Hq, Hkv, D, sum(nq) + D, behind=3, strided=nq == nk)
    scale = D ** -0.5
    o = torch.full((q.shape[0], Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    mq, mk = max(max(nq), 1), max(max(nk), 1)
    o, lse = api.bl_attn_forward(q, k, v, cq, ck, mq, mk, window, sinks, o=o)
    dq, dk, dv = (torch.full((t.shape[0], t.shape[1], D), 9.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v))
    api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, mq, mk, window, sinks, dq=dq, dk=dk, dv=dv)
    api.bl_check_device_error()
    for t, n in ((o, nq), (dq, nq), (dk, nk), (dv, nk)):
        assert bool((t[sum(n):] == 9.0).all())          # rows behind the last entry
    _compare(nq, nk, Hq, Hkv, D, window, sinks, scale, q, k, v, do, o, lse, (dq, dk, dv))
    again = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, mq, mk, window, sinks)
    assert torch.equal(again[0][:sum(nq)], dq[:sum(nq)])
    assert torch.equal(again[1][:sum(nk)], dk[:sum(nk)]) and torch.equal(again[2][:sum(nk)], dv[:sum(nk)])


def test_other_scale_and_large_scores():
    q, k, v, do, (cq, ck) = _inputs([300], [300], 2, 2, 64, 21)
    q *= 4
    o, lse = api.bl_attn_forward(q, k, v, cq, ck, 300, 300, scale=0.5)
    g = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, 300, 300, scale=0.5)
    _compare([300], [300], 2, 2, 64, 0, 0, 0.5, q, k, v, do, o, lse, g)


def test_neighbours_do_not_leak():
    """Infinities and NaN of one entry stay in it, although its rows share tiles with the next one's."""
    nq = [70, 90]
    q, k, v, do, (cq, ck) = _inputs(nq, nq, 2, 1, 64, 22)
    ref = api.bl_attn_forward(q, k, v, cq, ck, 90, 90)
    gref = api.bl_attn_backward(do, q, k, v, *ref, cq, ck, 90, 90)
    for t in (q, k, v, do):
        t[70:] = float("nan")
        t[75] = float("inf")
    got = api.bl_attn_forward(q, k, v, cq, ck, 90, 90)
    ggot = api.bl_attn_backward(do, q, k, v, *got, cq, ck, 90, 90)
    assert torch.equal(ref[0][:70], got[0][:70]) and torch.equal(ref[1][:, :70], got[1][:, :70])
    assert all(torch.equal(a[:70], b[:70]) for a, b in zip(gref, ggot))


def test_entry_longer_than_declared_is_reported():
    q, k, v, do, (cq, ck) = _inputs([300], [300], 1, 1, 64, 23)
    o, lse = api.bl_attn_forward(q, k, v, cq, ck, 100, 300)
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == 9
    bad = torch.tensor([0, 400], dtype=torch.int32).cuda()      # beyond the rows there are
    api.bl_attn_forward(q, k, v, bad, ck, 300, 300)
    with pytest.raises(api.BitLinearError):
        api.bl_check_device_error()


def test_capture_of_a_training_step():
    """Forward and backward captured while eager results of the same leaves live, then replayed on new values."""
    q, k, v, do, (cq, ck) = _inputs([150, 60], [150, 60], 4, 2, 64, 24)
    eager = api.bl_attn_forward(q, k, v, cq, ck, 150, 150, 64, 2)
    eager_g = api.bl_attn_backward(do, q, k, v, *eager, cq, ck, 150, 150, 64, 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = api.bl_attn_forward(q, k, v, cq, ck, 150, 150, 64, 2)
        grads = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, 150, 150, 64, 2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager[0]) and all(torch.equal(a, b) for a, b in zip(grads, eager_g))
    new = _inputs([150, 60], [150, 60], 4, 2, 64, 25)
    for t, n in zip((q, k, v, do), new):
        t.copy_(n)
    g.replay()
    torch.cuda.synchronize()
    _compare([150, 60], [150, 60], 4, 2, 64, 64, 2, 64 ** -0.5, q, k, v, do, o, lse, grads)


def test_window_and_sinks_beyond_every_length():
    q, k, v, do, (cq, ck) = _inputs([300, 40], [300, 40], 4, 2, 64, 26)
    o, lse = api.bl_attn_forward(q, k, v, cq, ck, 300, 300)
    g = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, 300, 300)
    for window, sinks in ((1 << 40, 0), (1 << 40, 1 << 50), (301, 0)):
        o2, lse2 = api.bl_attn_forward(q, k, v, cq, ck, 300, 300, window, sinks)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        g2 = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, 300, 300, window, sinks)
        assert all(torch.equal(a, b) for a, b in zip(g, g2))
    # a window with every key a sink hides nothing
    o2, lse2 = api.bl_attn_forward(q, k, v, cq, ck, 300, 300, 7, 1 << 40)
    g2 = api.bl_attn_backward(do, q, k, v, o2, lse2, cq, ck, 300, 300, 7, 1 << 40)
    _compare([300, 40], [300, 40], 4, 2, 64, 0, 0, 64 ** -0.5, q, k, v, do, o2, lse2, g2)


def test_long_sequence():
    """Many tiles, several waves of CTAs, sinks cut into pieces."""
    n = 2500
    q, k, v, do, (cq, ck) = _inputs([n], [n], 2, 1, 128, 27)
    for window, sinks in ((0, 0), (200, 5)):
        o, lse = api.bl_attn_forward(q, k, v, cq, ck, n, n, window, sinks)
        g = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, n, n, window, sinks)
        api.bl_check_device_error()
        _compare([n], [n], 2, 1, 128, window, sinks, 128 ** -0.5, q, k, v, do, o, lse, g)


def test_given_stream():
    """A call on a stream that is not the current one allocates there too: right whatever the current stream's pool
    hands out meanwhile."""
    q, k, v, do, (cq, ck) = _inputs([500, 300], [500, 300], 4, 2, 64, 28)
    o, lse = api.bl_attn_forward(q, k, v, cq, ck, 500, 500, 100, 3)
    g = api.bl_attn_backward(do, q, k, v, o, lse, cq, ck, 500, 500, 100, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    results = []
    for _ in range(6):
        o2, lse2 = api.bl_attn_forward(q, k, v, cq, ck, 500, 500, 100, 3, stream=side)
        results.append((o2, lse2, *api.bl_attn_backward(do, q, k, v, o2, lse2, cq, ck, 500, 500, 100, 3, stream=side)))
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        del junk
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, (o, lse, *g)))
