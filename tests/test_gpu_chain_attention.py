"""The operators together, as a server runs them: prompts through the ragged
attention into the cache, then token steps of a layer stack (DecodeChain with
a PagedKV) with forks, frees and a compaction in between."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api, workloads
from ternary_quantized_linear_bitlinear_b200.chain import PROJ, DecodeChain
from ternary_quantized_linear_bitlinear_b200.kv import PagedKV, rope_table
from _attention import EPS16, EPS32, attention, score_error, visible

pytestmark = pytest.mark.gpu

HIDDEN, FFN, HQ, HKV, D = 768, 2048, 12, 4, 64


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layers(n, seed=5):
    items = workloads.decode125m(seed=seed, M=1, layers=n)
    layers, gains = [], []
    for li in range(n):
        lay = {}
        for j, name in enumerate(PROJ):
            _, W, _ = items[li * len(PROJ) + j]
            lay[name] = (*api.bl_quant_weights(W.cuda()), W.shape[0], W.shape[1])
        layers.append(lay)
        gains.append((workloads.uniform((HIDDEN,), 0.9, 1.1, 30 + li).cuda(),
                      workloads.uniform((FFN,), 0.9, 1.1, 60 + li).cuda()))
    return layers, gains


def _rot(x, rope, pos):
    c, s = (t[:, None] for t in rope.double()[pos].split(D // 2, 1))
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _check_step(chain, history, rope, window, sinks, entries, lens):
    """Each layer's rotated q, new cache rows and attention output from that
    layer's own q, k, v as the GPU produced them; history[layer][seq] the
    float64 k, v rows of every earlier token (what the pages must hold)."""
    for li, b in enumerate(chain.layers):
        q, k, v = (b[n]["Y"].view(chain.M, -1, D).double().cpu() for n in ("q", "k", "v"))
        pos = torch.tensor([lens[s] - 1 if s >= 0 else 0 for s in entries])
        qr, kr = _rot(q, rope, pos), _rot(k, rope, pos)
        got_q = b["q_rot"].double().cpu()
        for m, s in enumerate(entries):
            if s < 0:
                continue
            assert bool(((got_q[m] - qr[m]).abs() <= 8 * EPS32 * q[m].abs().max()).all())
            hk, hv = history[li][s]
            hk.append(kr[m].float().bfloat16().double())
            hv.append(v[m].float().bfloat16().double())
            K, V = torch.stack(hk), torch.stack(hv)
            n = K.shape[0]
            assert n == lens[s]
            see = visible(1, n, window, sinks)
            for h in range(HQ):
                x = got_q[m, h][None]
                kh, vh = K[:, h // (HQ // HKV)], V[:, h // (HQ // HKV)]
                o, _, P = attention(x, kh, vh, see, D ** -0.5)
                d = score_error(x, kh, D ** -0.5, D).max().item()
                # a rotated key may round to bf16's other side of a tie that float32 does not resolve: one half
                # step of that key, in its score and weight
                d += EPS16 * 2.0 ** -8 * D ** -0.5 * (x.abs() @ kh.abs().T).max().item()
                rel = 2 * (d + 2.0 ** -21) + 2 * (n / 8 + 96) * 2.0 ** -23
                lim = rel * (P @ vh.abs()) + EPS32 * o.abs() + 1e-30
                got = b["attn"].view(chain.M, HQ, D)[m, h].double().cpu()
                assert bool(((got - o[0]).abs() <= lim[0]).all()), (li, m, h)


@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_serving_run(window, sinks):
    nl, M = 2, 4
    layers, gains = _layers(nl)
    kv = PagedKV(nl, 40, 8, HKV, D, 8, 12)
    rope = rope_table(96, D)
    seq_ids = _i32([0, 1, -1, -1])
    chain = DecodeChain(layers, gains, M, cache=kv, seq_ids=seq_ids, rope=rope, window=window, sinks=sinks)
    assert chain.launches_per_step() == 8 * nl + 1
    ropec = rope.cpu()

    # prompts of 13 and 5 tokens: q, k, v of each layer rotated, written and attended in one ragged batch
    g = torch.Generator().manual_seed(7)
    prompt = [13, 5]
    cu = _i32([0, 13, 18])
    assert kv.extend(_i32([0, 1]), _i32(prompt)).item() == 0
    history = [[([], []) for _ in range(8)] for _ in range(nl)]
    for li in range(nl):
        x = torch.randn(18, HQ + 2 * HKV, D, generator=g).cuda()
        q, k, v = kv.append(li, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], rope, cu, _i32([0, 1]), torch.bfloat16,
                            keep_kv=True)
        o, _ = api.bl_attn_forward(q, k, v, cu, cu, 13, 13, window, sinks)
        at = 0
        for s, n in enumerate(prompt):
            K, V = k[at:at + n].double().cpu(), v[at:at + n].double().cpu()
            history[li][s] = (list(K), list(V))
            # the prefill attention's last row is what the cache's attention gives for the same query
            one = kv.attend(li, q[at + n - 1][None], _i32([s]), window, sinks)
            diff = (one[0].float() - o[at + n - 1].float()).abs()
            assert bool((diff <= 3 * EPS16 * (o[at + n - 1].float().abs() + V.abs().max().item())).all())
            at += n
    lens = [13, 5] + [0] * 6

    gr = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()

    def fill():
        chain.x0.copy_(torch.randn(M, HIDDEN, generator=g).cuda() * 3)
        torch.cuda.synchronize()

    def advance(entries):
        for s in entries:
            if s >= 0:
                lens[s] += 1
        assert chain.status.item() == 0
        assert kv.lengths.tolist() == lens
        _check_step(chain, history, ropec, window, sinks, entries, lens)

    fill()
    chain.run(stream.cuda_stream)
    torch.cuda.synchronize()
    advance([0, 1, -1, -1])
    with torch.cuda.graph(gr, stream=stream):
        chain.run(stream.cuda_stream)

    def replay(entries):
        seq_ids.copy_(_i32(entries))
        fill()
        gr.replay()
        torch.cuda.synchronize()
        api.bl_check_device_error()
        advance(entries)

    replay([0, 1, -1, -1])
    # two forks of sequence 0 go on their own
    assert kv.fork(_i32([0, 0]), _i32([2, 5])).item() == 0
    lens[2] = lens[5] = lens[0]
    for li in range(nl):
        for s in (2, 5):
            history[li][s] = tuple(list(h) for h in history[li][0])
    for _ in range(3):
        replay([0, 1, 2, 5])
    # one ends, the pool is moved together, the rest go on
    kv.free(_i32([0]))
    lens[0] = 0
    used = int((kv.refs > 0).sum())
    assert kv.compact().item() == used and bool((kv.refs[used:] == 0).all())
    for _ in range(9):
        replay([5, -1, 1, 2])
    assert torch.isfinite(chain.out).all()


def test_a_step_without_pages_changes_nothing():
    layers, gains = _layers(1)
    kv = PagedKV(1, 2, 8, HKV, D, 2, 4)
    seq_ids = _i32([0, 1])
    chain = DecodeChain(layers, gains, 2, cache=kv, seq_ids=seq_ids, rope=rope_table(32, D))
    for _ in range(8):
        chain.run(torch.cuda.current_stream().cuda_stream)
    assert chain.status.item() == 0
    torch.cuda.synchronize()
    before = kv.pool.clone(), kv.tables.clone(), kv.lengths.clone(), kv.refs.clone(), chain.layers[0]["attn"].clone()
    chain.run(torch.cuda.current_stream().cuda_stream)
    assert chain.status.item() == 1
    for a, b in zip(before, (kv.pool, kv.tables, kv.lengths, kv.refs, chain.layers[0]["attn"])):
        assert torch.equal(a, b)
    api.bl_check_device_error()


def test_training_layer_gradients():
    """QAT of an attention block's projections with the library's forward and
    backward: q, k, v from BitLinear, rotation, attention, and the gradients
    back to the projections' inputs, against the same chain in float64 with
    straight-through quantizers."""
    lens = [50, 30]
    M, K = sum(lens), HIDDEN
    g = torch.Generator().manual_seed(11)
    X = torch.randn(M, K, generator=g).cuda()
    Ws = [workloads.normal((h * D, K), 0.02, 80 + i).cuda() for i, h in enumerate((HQ, HKV, HKV))]
    dO = torch.randn(M, HQ, D, generator=g).bfloat16().cuda()
    rope, cu = rope_table(64, D), _i32([0, 50, 80])
    packs = [api.bl_quant_weights(W) for W in Ws]
    x_q, s = api.bl_quant_act(X)
    Y = [api.bl_forward(p, gm, x_q, s, W.shape[0]) for (p, gm), W in zip(packs, Ws)]
    q, k, v = api.bl_rope_append(*(y.view(M, -1, D) for y in Y), rope=rope, cu_seqlens=cu, out_dtype=torch.bfloat16)
    o, lse = api.bl_attn_forward(q, k, v, cu, cu, 50, 50, 16, 2)
    grads = api.bl_attn_backward(dO, q, k, v, o, lse, cu, cu, 50, 50, 16, 2)
    dq, dk, _ = api.bl_rope_append(grads[0], grads[1], grads[2], rope=rope, cu_seqlens=cu, inverse=True)
    dY = [dq.reshape(M, -1), dk.reshape(M, -1), grads[2].reshape(M, -1)]
    dX = sum(api.bl_backward_dx(d, p, gm, K) for d, (p, gm) in zip(dY, packs))
    api.bl_check_device_error()

    # float64, the quantized operands as they are, gradients by differentiation
    xs = (x_q.double() / s.double()[:, None]).cpu().requires_grad_()
    ws = []
    for (p, gm), W in zip(packs, Ws):
        r = (W / gm).round().clamp(-1, 1)
        ws.append((r.double() * gm.double()).cpu())
    qkv = [(xs @ w.T).view(M, -1, D) for w in ws]
    pos = torch.cat([torch.arange(n) for n in lens])
    qr, kr = _rot(qkv[0], rope.cpu(), pos), _rot(qkv[1], rope.cpu(), pos)
    outs, at = [], 0
    for n in lens:
        see = visible(n, n, 16, 2)
        outs.append(torch.stack([attention(qr[at:at + n, h], kr[at:at + n, h // 3], qkv[2][at:at + n, h // 3], see,
                                           D ** -0.5)[0] for h in range(HQ)], 1))
        at += n
    torch.cat(outs).backward(dO.double().cpu())
    # bfloat16 along the way (q, k, v, P, dS, the gradients and their rotation: seven roundings of half a step each
    # on independent terms), against the norm of the whole
    ref = xs.grad
    err = (dX.double().cpu() - ref).norm() / ref.norm()
    assert err < 7 * EPS16, err
