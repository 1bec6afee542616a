"""The page tables' entry points against the same bookkeeping on lists, and
the pages they copy."""
from __future__ import annotations

import random

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api
from ternary_quantized_linear_bitlinear_b200.kv import PagedKV
from _attention import PageModel

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pair(pages, ps, seqs, cols, layers=2, Hkv=2, D=16, dtype=torch.bfloat16, seed=0):
    kv = PagedKV(layers, pages, ps, Hkv, D, seqs, cols, dtype)
    kv.pool.copy_(torch.randn(kv.pool.shape, generator=torch.Generator().manual_seed(seed)).to(dtype))
    return kv, PageModel(pages, ps, seqs, cols)


@pytest.mark.parametrize("pages,ps,seqs,cols,dtype", [(40, 16, 9, 6, torch.bfloat16), (3000, 8, 200, 40, torch.float32),
                                                      (5, 64, 3, 2, torch.bfloat16)])
def test_random_runs(pages, ps, seqs, cols, dtype):
    kv, model = _pair(pages, ps, seqs, cols, dtype=dtype, seed=pages)
    rng = random.Random(pages)
    data = kv.pool.clone()
    seen = set()
    for step in range(60):
        op = rng.choice(["extend", "extend", "extend", "free", "fork", "fork", "compact"])
        if op == "extend":
            ids = rng.sample(range(seqs), rng.randint(1, min(seqs, 20)))
            counts = [rng.choice([0, 1, 1, rng.randrange(ps * cols // 2 + 1)]) for _ in ids]
            ids = [i if rng.random() < 0.9 else -1 for i in ids]
            active = torch.full((len(ids),), 99, dtype=torch.int32, device="cuda")
            st = kv.extend(_i32(ids), _i32(counts), active=active).item()
            want = model.extend(ids, counts)
            assert st == want
            assert active.tolist() == (ids if st == 0 else [-1] * len(ids))
            seen.add(("extend", st))
        elif op == "free":
            ids = [rng.randrange(-1, seqs) for _ in range(rng.randint(1, 12))]   # repeats and empty ones among them
            kv.free(_i32(ids))
            model.free(dict.fromkeys(ids))
        elif op == "fork":
            n = rng.randint(1, min(6, seqs // 2))
            ids = rng.sample(range(seqs), 2 * n)
            src, dst = ids[:n], ids[n:]
            if rng.random() < 0.7:
                empty = [i for i in range(seqs) if model.lengths[i] == 0][:n]
                src = [rng.choice([i for i in range(seqs) if i not in empty] or [-1]) for _ in empty]
                dst = empty
            if not dst:
                continue
            st = kv.fork(_i32(src), _i32(dst)).item()
            assert st == model.fork(src, dst)
            seen.add(("fork", st))
            if st == 0:
                for a, b in model.moves:
                    data[:, :, b] = data[:, :, a]
        else:
            assert kv.compact().item() == model.compact()
            for a, b in model.moves:
                data[:, :, b] = data[:, :, a]
        model.check(kv.tables, kv.lengths, kv.refs)
        assert torch.equal(kv.pool, data)
    api.bl_check_device_error()
    assert ("extend", 0) in seen


def test_statuses():
    kv, model = _pair(6, 16, 4, 4)
    def both(op, *a):
        got = getattr(kv, op)(*[_i32(x) for x in a]).item()
        assert got == getattr(model, op)(*a)
        model.check(kv.tables, kv.lengths, kv.refs)
        return got
    assert both("extend", [0, 1], [33, 16]) == 0          # 3 + 1 pages of 6
    assert both("extend", [2, 1], [17, 17]) == 1          # 2 + 2 more: too few, nothing changes
    assert both("extend", [0], [32]) == 2                 # 65 tokens do not fit four pages
    assert both("extend", [0, 0], [1, 1]) == 3            # twice
    assert both("extend", [4], [1]) == 3
    assert both("extend", [0], [-1]) == 3
    assert both("extend", [2], [0]) == 0                  # nothing to do
    assert both("extend", [-1, 2], [500, 1]) == 0         # padding's count does not matter
    assert both("fork", [0], [1]) == 3                    # not empty
    assert both("fork", [0, 1], [3, 3]) == 3
    assert both("fork", [0, 3], [3, 0]) == 3              # a source that is a target
    assert both("fork", [0], [9]) == 3
    assert both("fork", [0], [3]) == 0                    # takes the last page
    kv.free(_i32([1]))
    model.free([1])
    assert both("fork", [1], [1]) == 3
    kv.free(_i32([2, 3, 2]))
    model.free([2, 3])
    model.check(kv.tables, kv.lengths, kv.refs)
    # too few pages for the partial pages of two forks
    kv2, m2 = _pair(3, 8, 4, 4)
    for k, m in ((kv2, m2),):
        k.extend(_i32([0]), _i32([12]))
        m.extend([0], [12])
        assert k.fork(_i32([0, 0]), _i32([1, 2])).item() == m.fork([0, 0], [1, 2]) == 1
        m.check(k.tables, k.lengths, k.refs)
    # an id beyond the tables is reported
    kv.free(_i32([7]))
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == 9


def test_large_pool_and_many_entries():
    kv, model = _pair(70000, 8, 3000, 30, layers=1, Hkv=1, D=16)
    rng = random.Random(4)
    ids = list(range(2500))
    rng.shuffle(ids)
    counts = [rng.randrange(0, 200) for _ in ids]
    assert kv.extend(_i32(ids), _i32(counts)).item() == model.extend(ids, counts) == 0
    gone = ids[::3]
    kv.free(_i32(gone))
    model.free(gone)
    data = kv.pool.clone()
    assert kv.compact().item() == model.compact()
    a, b = (torch.tensor(x, device="cuda") for x in zip(*model.moves))
    data[:, :, b] = data[:, :, a]
    model.check(kv.tables, kv.lengths, kv.refs)
    assert torch.equal(kv.pool, data)
    src, dst = [i for i in ids if i not in set(gone)][:400], list(range(2500, 2900))
    assert kv.fork(_i32(src), _i32(dst)).item() == model.fork(src, dst) == 0
    a, b = (torch.tensor(x, device="cuda") for x in zip(*model.moves))
    data[:, :, b] = data[:, :, a]
    model.check(kv.tables, kv.lengths, kv.refs)
    assert torch.equal(kv.pool, data)


def test_captured_steps():
    kv, model = _pair(64, 16, 8, 8)
    ids, counts = _i32([0, 5, 2]), _i32([3, 20, 1])
    src, dst, gone = _i32([0]), _i32([6]), _i32([6])
    st = torch.zeros(2, 4, dtype=torch.int32, device="cuda")

    def step():
        kv.free(gone)
        kv.extend(ids, counts, st[0])
        kv.fork(src, dst, st[1])

    def ref():
        model.free([6])
        return model.extend([0, 5, 2], counts.tolist()), model.fork([0], [6])

    step()
    assert ref() == (0, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    model.check(kv.tables, kv.lengths, kv.refs)
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert ref() == (st[0, 0].item(), st[1, 0].item())
        model.check(kv.tables, kv.lengths, kv.refs)


def test_a_table_that_names_no_page_is_reported():
    kv, _ = _pair(8, 8, 4, 4)
    kv.extend(_i32([0]), _i32([12]))
    kv.tables[0, 1] = -1
    assert kv.fork(_i32([0]), _i32([1])).item() == 0
    with pytest.raises(api.BitLinearError) as e:
        api.bl_check_device_error()
    assert e.value.status == 9
    kv.tables[0, 0] = 10 ** 6
    kv.fork(_i32([0]), _i32([2]))
    with pytest.raises(api.BitLinearError):
        api.bl_check_device_error()
    kv.free(_i32([0]))
    with pytest.raises(api.BitLinearError):
        api.bl_check_device_error()


def test_given_stream():
    kv, model = _pair(64, 8, 8, 8)
    side = torch.cuda.Stream()
    ids, counts = _i32([0, 3]), _i32([20, 9])
    torch.cuda.synchronize()
    data = kv.pool.clone()
    torch.cuda.synchronize()
    st = [kv.extend(ids, counts, stream=side), kv.fork(ids, _i32([1, 2]), stream=side)]
    kv.free(_i32([0]), stream=side)
    n = kv.compact(stream=side)
    torch.cuda.synchronize()
    model.extend([0, 3], [20, 9])
    model.fork([0, 3], [1, 2])
    for a, b in model.moves:
        data[:, :, b] = data[:, :, a]
    model.free([0])
    assert n.item() == model.compact() and [s.item() for s in st] == [0, 0]
    for a, b in model.moves:
        data[:, :, b] = data[:, :, a]
    model.check(kv.tables, kv.lengths, kv.refs)
    assert torch.equal(kv.pool, data)
