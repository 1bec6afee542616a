"""bl_rope_append against a plain 64-bit rotation, and what it must not touch."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api
from ternary_quantized_linear_bitlinear_b200.kv import rope_table
from _attention import EPS16, EPS32

pytestmark = pytest.mark.gpu


def _rotate(x, rope, pos, inverse=False):
    """x [T, H, D] float64 -> (rotated, sum of the terms' magnitudes)."""
    D = x.shape[-1]
    c, s = (t[:, None] for t in rope.double()[pos].split(D // 2, 1))
    s = -s if inverse else s
    a, b = x[..., :D // 2], x[..., D // 2:]
    y = torch.cat([a * c - b * s, b * c + a * s], -1)
    mag = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    return y, mag


def _close(out, ref, mag):
    """Two products and a sum in float32 (at most three roundings of the terms'
    magnitudes), then one rounding to the output type."""
    half = EPS16 if out.dtype == torch.bfloat16 else EPS32
    err = (out.double().cpu() - ref).abs()
    lim = 3 * EPS32 * mag + half * (ref.abs() + 3 * EPS32 * mag)
    assert bool((err <= lim).all()), (err - lim).max()


@pytest.mark.parametrize("src,odt,cdt", [(torch.float32, torch.float32, torch.bfloat16),
                                         (torch.float32, torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(12, 4, 64, 16), (5, 5, 128, 8), (8, 1, 16, 64), (6, 2, 80, 32)])
def test_ragged_append(src, odt, cdt, Hq, Hkv, D, ps):
    g = torch.Generator().manual_seed(D + Hq)
    new, past, seqs = [1, 37, 0, 8, 130], [0, 11, 5, 2 * ps, ps - 1], [4, 0, 2, 6, 1]
    T, extra = sum(new), 3                       # three rows behind the last entry
    max_seqs, max_pages = 7, -(-200 // ps)
    lengths = torch.zeros(max_seqs, dtype=torch.int32)
    for n, b, s in zip(new, past, seqs):
        lengths[s] = n + b
    need = [-(-int(x) // ps) for x in lengths]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).tolist()
    tables = torch.full((max_seqs, max_pages), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    # q, k, v are columns of one projection output
    qkv = torch.randn(T + extra, Hq + 2 * Hkv, D, generator=g).to(src).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    rope = rope_table(256, D)
    kp = torch.randn(pages, Hkv, ps, D, generator=g).to(cdt)
    vp = torch.randn(pages, Hkv, ps, D, generator=g).to(cdt)
    kd, vd = kp.cuda(), vp.cuda()
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32).cuda()
    q_out = torch.full((T + extra, Hq, D), 7.0, dtype=odt, device="cuda")
    k_out = torch.full((T + extra, Hkv, D), 7.0, dtype=odt, device="cuda")
    v_out = torch.full((T + extra, Hkv, D), 7.0, dtype=odt, device="cuda")
    api.bl_rope_append(q, k, v, rope, cu, lengths.cuda(), torch.tensor(seqs, dtype=torch.int32).cuda(), kd, vd,
                       tables.cuda(), out_dtype=odt, q_out=q_out, k_out=k_out, v_out=v_out)
    api.bl_check_device_error()
    pos = torch.tensor([past[b] + i for b in range(len(new)) for i in range(new[b])])
    seq = torch.tensor([seqs[b] for b in range(len(new)) for _ in range(new[b])])
    rq, mq = _rotate(q[:T].double().cpu(), rope.cpu(), pos)
    rk, mk = _rotate(k[:T].double().cpu(), rope.cpu(), pos)
    _close(q_out[:T], rq, mq)
    _close(k_out[:T], rk, mk)
    assert torch.equal(v_out[:T], v[:T].to(odt))
    for t in (q_out, k_out, v_out):
        assert bool((t[T:] == 7.0).all())        # rows behind the last entry
    page, slot = tables[seq, pos // ps].long(), pos % ps
    _close(kd.cpu()[page, :, slot], rk, mk)
    assert torch.equal(vd.cpu()[page, :, slot], v[:T].to(cdt).cpu())
    # everything else in the pages as it was
    touched = torch.zeros(pages, ps, dtype=torch.bool)
    touched[page, slot] = True
    keep = ~touched[:, None, :, None].expand_as(kp)
    assert torch.equal(kd.cpu()[keep], kp[keep]) and torch.equal(vd.cpu()[keep], vp[keep])


def test_rotation_without_cache_and_its_inverse():
    T, H, D = 50, 3, 64
    x = torch.randn(T, H, D, generator=torch.Generator().manual_seed(1)).cuda()
    rope = rope_table(T, D)
    cu = torch.tensor([0, 20, T], dtype=torch.int32).cuda()
    y, _, _ = api.bl_rope_append(x, rope=rope, cu_seqlens=cu)
    pos = torch.cat([torch.arange(20), torch.arange(30)])
    ref, mag = _rotate(x.double().cpu(), rope.cpu(), pos)
    _close(y, ref, mag)
    # the gradient: rotating back; in place
    z, _, _ = api.bl_rope_append(y, rope=rope, cu_seqlens=cu, q_out=y, inverse=True)
    assert z.data_ptr() == y.data_ptr()
    ref, mag = _rotate(ref, rope.cpu(), pos, inverse=True)
    # y's own error passes through the rotation once more
    err = (z.double().cpu() - x.double().cpu()).abs()
    assert bool((err <= 10 * EPS32 * (mag + x.double().cpu().abs())).all())
    # k and v alone; no rotation: a copy
    k, v = x[:, :2], x[:, 1:]
    _, k2, v2 = api.bl_rope_append(k=k, v=v, out_dtype=torch.bfloat16)
    assert torch.equal(k2, k.bfloat16()) and torch.equal(v2, v.bfloat16())


def test_bad_indexes_write_nothing_and_are_reported():
    D, ps = 32, 8
    kp = torch.zeros(4, 1, ps, D, device="cuda")
    x = torch.randn(1, 1, D, device="cuda")
    rope = rope_table(16, D)

    def call(lengths, table, ids):
        out = torch.full((1, 1, D), 3.0, device="cuda")
        k, v = kp.clone(), kp.clone()
        i32 = dict(dtype=torch.int32, device="cuda")
        api.bl_rope_append(x, x, x, rope, None, torch.tensor(lengths, **i32), torch.tensor([ids], **i32), k, v,
                           torch.tensor(table, **i32), q_out=out)
        try:
            api.bl_check_device_error()
            bad = False
        except api.BitLinearError as e:
            assert e.status == 9
            bad = True
        return bad, bool((k != 0).any() or (v != 0).any()), bool((out != 3.0).any())

    good = [[0, 1], [2, 3]]
    assert call([3, 9], good, 1) == (False, True, True)
    assert call([3, 9], good, -1) == (False, False, False)     # padding: no error, nothing written
    assert call([3, 9], good, 2) == (True, False, False)       # no such sequence
    assert call([0, 9], good, 0) == (True, False, False)       # not extended: position -1
    assert call([17, 9], good, 0) == (True, False, False)      # beyond the rope and the table
    assert call([3, 9], [[4, 1], [2, 3]], 0)[:2] == (True, False)   # no such page
    assert call([3, 9], [[-1, 1], [2, 3]], 0)[:2] == (True, False)
