"""bl_attn_decode against plain 64-bit attention over the gathered pages."""
from __future__ import annotations

import math

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api
from _attention import EPS16, EPS32, attention, score_error

pytestmark = pytest.mark.gpu


def _cache(lens, ps, Hkv, D, dtype, seed, fill=float("nan"), spare=0):
    """Pages in a scrambled order; what lies behind a length holds `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g).tolist()
    tables = torch.full((len(lens), max(need + [1]) + spare), -1, dtype=torch.int32)
    kp = torch.full((pages, Hkv, ps, D), fill)
    vp = torch.full((pages, Hkv, ps, D), fill)
    ks, vs, at = [], [], 0
    for s, n in enumerate(lens):
        tables[s, :need[s]] = torch.tensor(order[at:at + need[s]], dtype=torch.int32)
        at += need[s]
        k, v = (torch.randn(n, Hkv, D, generator=g).to(dtype).float() for _ in "kv")
        ks.append(k.double())
        vs.append(v.double())
        j = torch.arange(n)
        page = tables[s].long()[j // ps]
        kp[page, :, j % ps] = k
        vp[page, :, j % ps] = v
    return kp.to(dtype).cuda(), vp.to(dtype).cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), ks, vs


def _check(out, lse, q, ks, vs, entries, window, sinks, scale):
    """entries: the sequence of each row, None for one that is to stay as it was.

    Bound: a score is off by d (score_error), so a weight by d + 2^-21 (exp2 to
    2 ulp, its argument's rounding, the two rescalings of a partial) relative;
    numerator and denominator carry that and one rounding per addition on a
    term's way (at most one in 8 keys plus the joins), the output type's half
    step comes on top."""
    B, H, D = q.shape
    group = H // ks[0].shape[1]
    half = EPS16 if out.dtype == torch.bfloat16 else EPS32
    for b, s in enumerate(entries):
        if s is None:
            continue
        n = ks[s].shape[0]
        j = torch.arange(n)
        see = ((j >= n - window) | (j < sinks))[None] if window else torch.ones(1, n, dtype=torch.bool)
        for h in range(H):
            k, v = ks[s][:, h // group], vs[s][:, h // group]
            x = q[b, h].double().cpu()[None]
            o, l, P = attention(x, k, v, see, scale)
            if n == 0:
                assert bool((out[b, h] == 0).all()) and lse[b, h].item() == -math.inf
                continue
            d = torch.where(see, score_error(x, k, scale, D), 0.0).max().item()
            rel = 2 * (d + 2.0 ** -21) + 2 * (n / 8 + 96) * 2.0 ** -23
            lim = rel * (P @ v.abs()) + half * (o.abs() + rel * (P @ v.abs()))
            err = (out[b, h].double().cpu() - o[0]).abs()
            assert bool((err <= lim[0]).all()), (b, h, (err / lim[0]).max())
            assert abs(lse[b, h].item() - l.item()) <= rel + 4 * EPS32 * (abs(l.item()) + 1)


CASES = [
    # Hq, Hkv, D, page, window, sinks
    (12, 4, 64, 16, 0, 0),
    (12, 4, 128, 8, 100, 5),
    (20, 20, 128, 32, 0, 0),
    (8, 1, 64, 64, 64, 0),
    (16, 1, 80, 16, 0, 0),      # a group of 16: two head groups
    (11, 1, 128, 128, 30, 40),  # 6 + 5 heads; more sinks than window
    (5, 5, 16, 8, 7, 1),
    (6, 2, 32, 1024, 1, 0),
    (24, 8, 96, 16, 33, 100),
]


@pytest.mark.parametrize("src,cache", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("Hq,Hkv,D,ps,window,sinks", CASES)
def test_ragged_batch(src, cache, Hq, Hkv, D, ps, window, sinks):
    lens = [1, 0, 17, 128, 8, 333, 2, 64, 1025, 15]
    kp, vp, tables, lengths, ks, vs = _cache(lens, ps, Hkv, D, cache, Hq * D + ps)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(3)).to(src).cuda()
    out, lse = api.bl_attn_decode(q, kp, vp, tables, lengths, window=window, sinks=sinks, return_lse=True)
    api.bl_check_device_error()
    _check(out, lse, q, ks, vs, range(len(lens)), window, sinks, D ** -0.5)
    # the same inputs give the same bits
    again, lse2 = api.bl_attn_decode(q, kp, vp, tables, lengths, window=window, sinks=sinks, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float32])
def test_long_sequence_is_split_and_joined(cache):
    kp, vp, tables, lengths, ks, vs = _cache([20011], 64, 2, 64, cache, 5)
    q = (torch.randn(1, 6, 64, generator=torch.Generator().manual_seed(4)) * 3).cuda()
    out, lse = api.bl_attn_decode(q, kp, vp, tables, lengths, scale=0.2, return_lse=True)
    _check(out, lse, q, ks, vs, [0], 0, 0, 0.2)


def test_sequence_ids_padding_and_strided_queries():
    lens = [40, 7, 300, 0]
    kp, vp, tables, lengths, ks, vs = _cache(lens, 16, 2, 64, torch.bfloat16, 8, spare=3)
    wide = torch.randn(6, 4 + 5, 64, generator=torch.Generator().manual_seed(9)).cuda()
    q = wide[:, 3:7]                                    # four heads of a wider row
    ids = torch.tensor([2, -1, 0, 2, -1, 3], dtype=torch.int32).cuda()
    out = torch.full((6, 4, 64), 5.0, device="cuda")
    lse = torch.full((6, 4), 5.0, device="cuda")
    api.bl_attn_decode(q, kp, vp, tables, lengths, ids, out=out, lse=lse)
    api.bl_check_device_error()
    _check(out, lse, q, ks, vs, [2, None, 0, 2, None, 3], 0, 0, 64 ** -0.5)
    for b in (1, 4):
        assert bool((out[b] == 5.0).all() and (lse[b] == 5.0).all())
    # more entries than CTA threads, most of them padding
    many = torch.full((700,), -1, dtype=torch.int32)
    many[::50] = 2
    big = torch.randn(700, 4, 64, generator=torch.Generator().manual_seed(10)).cuda()
    o = torch.full((700, 4, 64), 5.0, device="cuda")
    l2 = torch.full((700, 4), 5.0, device="cuda")
    api.bl_attn_decode(big, kp, vp, tables, lengths, many.cuda(), out=o, lse=l2)
    api.bl_check_device_error()
    _check(o, l2, big, ks, vs, [2 if i % 50 == 0 else None for i in range(700)], 0, 0, 64 ** -0.5)
    assert bool((o[1:50] == 5.0).all())


def test_bad_pages_and_ids_are_skipped_and_reported():
    kp, vp, tables, lengths, ks, vs = _cache([40, 40], 16, 1, 32, torch.bfloat16, 11)
    q = torch.randn(2, 1, 32, generator=torch.Generator().manual_seed(12)).cuda()
    broken = tables.clone()
    broken[0, 1] = 10 ** 6
    out, lse = api.bl_attn_decode(q, kp, vp, broken, lengths, return_lse=True)
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == 9
    # the page's 16 keys are left out, the other entry is whole
    keep = torch.tensor([i for i in range(40) if not 16 <= i < 32])
    _check(out[:1], lse[:1], q[:1], [ks[0][keep]], [vs[0][keep]], [0], 0, 0, 32 ** -0.5)
    _check(out[1:], lse[1:], q[1:], ks, vs, [1], 0, 0, 32 ** -0.5)
    for ids, lens in (([0, 2], [40, 40]), ([0, 1], [40, 2000])):
        api.bl_attn_decode(q, kp, vp, tables, torch.tensor(lens, dtype=torch.int32).cuda(),
                           torch.tensor(ids, dtype=torch.int32).cuda())
        with pytest.raises(api.BitLinearError) as e:
            api.bl_check_device_error()
        assert e.value.status == 9
    api.bl_attn_decode(q, kp, vp, tables, lengths)
    api.bl_check_device_error()


def test_captured_and_replayed_with_new_lengths():
    lens = [900, 33]
    kp, vp, tables, lengths, ks, vs = _cache(lens, 32, 4, 64, torch.bfloat16, 13)
    q = torch.randn(2, 12, 64, generator=torch.Generator().manual_seed(14)).cuda()
    out, lse = torch.empty_like(q), torch.empty(2, 12, device="cuda")
    api.bl_attn_decode(q, kp, vp, tables, lengths, out=out, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.bl_attn_decode(q, kp, vp, tables, lengths, out=out, lse=lse)
    for new in ([900, 33], [1, 20], [512, 0]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, q, [k[:n] for k, n in zip(ks, new)], [v[:n] for v, n in zip(vs, new)], [0, 1], 0, 0, 64 ** -0.5)


def test_two_streams_at_once():
    kp, vp, tables, lengths, ks, vs = _cache([3000, 500, 1], 16, 2, 128, torch.bfloat16, 15)
    q = torch.randn(3, 6, 128, generator=torch.Generator().manual_seed(16)).cuda()
    ref = api.bl_attn_decode(q, kp, vp, tables, lengths)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(api.bl_attn_decode(q, kp, vp, tables, lengths))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie beyond 2^32 of the pool's start."""
    ps, Hkv, D = 64, 4, 128
    pages = (1 << 32) // (ps * Hkv * D * 2) + 40
    kp = torch.zeros(pages, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    ids = list(range(pages - 5, pages))
    g = torch.Generator().manual_seed(17)
    k, v = (torch.randn(5, Hkv, ps, D, generator=g).bfloat16() for _ in "kv")
    kp[ids], vp[ids] = k.cuda(), v.cuda()
    tables = torch.tensor([ids], dtype=torch.int32).cuda()
    lengths = torch.tensor([300], dtype=torch.int32).cuda()
    q = torch.randn(1, 4, D, generator=g).cuda()
    out, lse = api.bl_attn_decode(q, kp, vp, tables, lengths, return_lse=True)
    flat = [t.transpose(1, 2).reshape(5 * ps, Hkv, D)[:300].double() for t in (k, v)]
    _check(out, lse, q, [flat[0]], [flat[1]], [0], 0, 0, D ** -0.5)
    # and the append writes there
    x = torch.randn(1, Hkv, D, generator=g).cuda()
    api.bl_rope_append(k=x, v=x, lengths=lengths, k_pages=kp, v_pages=vp, tables=tables)
    assert torch.equal(kp[ids[4], :, 299 % ps], x[0].bfloat16())


def test_given_stream_and_large_values_of_everything():
    kp, vp, tables, lengths, ks, vs = _cache([300, 70], 16, 2, 64, torch.bfloat16, 18)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(19)).cuda()
    ref = api.bl_attn_decode(q, kp, vp, tables, lengths)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [api.bl_attn_decode(q, kp, vp, tables, lengths, window=w, sinks=s, stream=side)
            for w, s in ((0, 0), (1 << 40, 0), (0, 1 << 40), (300, 1 << 50), (1, 1 << 40))]
    torch.cuda.synchronize()
    for o in outs[:4]:
        assert torch.equal(o, ref)
    _check(outs[4], torch.zeros(2, 4), q, ks, vs, [], 0, 0, 0.125)
    assert (outs[4] - ref).abs().max() < 1e-5       # every key is a sink: the same keys, perhaps in other batches
    # lengths no table can hold, for many entries: cut off and reported
    huge = torch.full((2,), 2 ** 31 - 1, dtype=torch.int32).cuda()
    api.bl_attn_decode(q.repeat(300, 1, 1), kp, vp, tables, huge, torch.zeros(600, dtype=torch.int32).cuda())
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == 9
