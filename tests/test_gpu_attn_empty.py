"""Single-token attention of batches with empty sequences: their rows, and their cost."""
from __future__ import annotations

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api

pytestmark = pytest.mark.gpu


def _cache(lens, Hkv, D, ps, dtype):
    cols = max(1, max(-(-n // ps) for n in lens))
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    tables = torch.arange(len(lens) * cols, dtype=torch.int32).view(len(lens), cols)
    k, v = (torch.randn(len(lens) * cols, Hkv, ps, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    return k, v, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


@pytest.mark.parametrize("B", [1, 5, 300])
@pytest.mark.parametrize("Hq,Hkv,D,qt,kt", [(4, 2, 64, torch.float32, torch.bfloat16), (3, 1, 128, torch.bfloat16, torch.bfloat16),
                                            (6, 2, 16, torch.bfloat16, torch.float32), (20, 20, 80, torch.float32, torch.float32)])
def test_rows_of_empty_sequences(B, Hq, Hkv, D, qt, kt):
    """0 and -inf for them, padded entries as they were, the others as in a batch without any of these."""
    lens = [(7 * i) % 90 if i % 3 == 1 else 0 for i in range(B)]
    k, v, tables, lengths = _cache(lens, Hkv, D, 16, kt)
    ids = torch.tensor([-1 if i % 5 == 4 else i for i in range(B)], dtype=torch.int32).cuda()
    q = torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(1)).to(qt).cuda()
    out, lse = torch.full_like(q, 9.0), torch.full((B, Hq), 9.0, device="cuda")
    api.bl_attn_decode(q, k, v, tables, lengths, ids, out=out, lse=lse)
    api.bl_check_device_error()
    for i in range(B):
        if i % 5 == 4:
            assert bool((out[i] == 9.0).all()) and bool((lse[i] == 9.0).all())
        elif lens[i] == 0:
            assert bool((out[i] == 0.0).all()) and bool((lse[i] == -torch.inf).all())
        else:
            assert bool(out[i].isfinite().all()) and bool((out[i] != 9.0).any())
            page = tables[i].long()
            kk, vv = (t[page].transpose(0, 1).flatten(1, 2)[:, :lens[i]].double().repeat_interleave(Hq // Hkv, 0) for t in (k, v))
            s = torch.einsum("hd,hjd->hj", q[i].double(), kk) * D ** -0.5
            ref = torch.einsum("hj,hjd->hd", s.softmax(-1), vv)
            # (an output is rounded by 2^-8 of at most the largest value; as much again is far above the rest)
            assert bool(((out[i] - ref).abs() <= 2.0 ** -7 * vv.abs().amax((0, 1))).all())


def test_cost_of_an_empty_sequence():
    """A batch in which some sequences are empty takes no longer than the full one (20 heads of 128)."""
    B = 64

    def best(lens):
        k, v, tables, _ = _cache([1024] * B, 20, 128, 32, torch.bfloat16)
        lengths = torch.tensor(lens, dtype=torch.int32).cuda()
        q = torch.randn(B, 20, 128, device="cuda")
        times = []
        for _ in range(30):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            ev[0].record()
            api.bl_attn_decode(q, k, v, tables, lengths)
            ev[1].record()
            torch.cuda.synchronize()
            times.append(ev[0].elapsed_time(ev[1]))
        return min(times)

    full = best([1024] * B)
    for empty in (1, 8):
        some = best([0 if i % (B // empty) == 3 else 1024 for i in range(B)])
        assert some <= 1.15 * full, (some, full)
