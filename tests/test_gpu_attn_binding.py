"""The compiled way to the attention calls: what it takes, what it leaves to
the Python checks, and that both ways give the same bits.

Refusals run with entry points that only count their calls, so that no bad
argument reaches a kernel."""
from __future__ import annotations

import ctypes

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api, build
from ternary_quantized_linear_bitlinear_b200.kv import rope_table

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAMES = {"rope_append": "q k v rope cu_seqlens lengths seq_ids k_pages v_pages tables out_dtype q_out k_out v_out keep_kv inverse",
         "attn_decode": "q k_pages v_pages tables lengths seq_ids window sinks scale out lse return_lse workspace",
         "kv_extend": "tables lengths refs seq_ids counts page_size status active",
         "kv_free": "tables lengths refs seq_ids page_size",
         "kv_fork": "pool tables lengths refs src dst status workspace",
         "kv_compact": "pool tables refs n_live workspace",
         "attn_forward": "q k v cu_q cu_k max_q max_k window sinks scale o lse",
         "attn_backward": "do q k v o lse cu_q cu_k max_q max_k window sinks scale dq dk dv workspace"}
NAMES = {f: names.split() for f, names in NAMES.items()}


def calls(dev):
    """One plain valid call of each function."""
    g = torch.Generator().manual_seed(11)

    def rnd(*shape, dtype=BF):
        return torch.randn(*shape, generator=g).to(dtype).to(dev)

    def i32(*values):
        return torch.tensor(values, dtype=I32, device=dev)

    Hq, Hkv, D, ps = 4, 2, 64, 16
    tables = torch.full((3, 4), -1, dtype=I32, device=dev)
    tables[0, :2] = i32(0, 1)
    tables[1, :1] = i32(2)
    lengths = i32(20, 9, 0)
    refs = i32(1, 1, 1, 0, 0, 0)
    k_pages, v_pages = rnd(6, Hkv, ps, D), rnd(6, Hkv, ps, D)
    pool = rnd(2, 6, Hkv, ps, D)
    q, k, v, do = rnd(7, Hq, D), rnd(9, Hkv, D), rnd(9, Hkv, D), rnd(7, Hq, D)
    cu_q, cu_k = i32(0, 3, 7), i32(0, 4, 9)
    tq, tk = rnd(2, Hq, D, dtype=F32), rnd(2, Hkv, D, dtype=F32)
    cache = dict(k_pages=k_pages, v_pages=v_pages, tables=tables, lengths=lengths)
    table = dict(tables=tables, lengths=lengths, refs=refs)
    ragged = dict(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, max_q=4, max_k=5, window=3, sinks=1, scale=None)
    o = rnd(7, Hq, D)
    lse = rnd(Hq, 7, dtype=F32)
    return {
        "rope_append": dict(q=tq, k=tk, v=tk.clone(), rope=rope_table(64, D, device=dev), seq_ids=i32(0, 1), out_dtype=BF,
                            keep_kv=True, inverse=False, **cache),
        "attn_decode": dict(q=tq, seq_ids=i32(1, 0), window=0, sinks=0, scale=0.1, return_lse=True, **cache),
        "kv_extend": dict(seq_ids=i32(0, 2), counts=i32(13, 1), page_size=ps, active=i32(0, 0), **table),
        "kv_free": dict(seq_ids=i32(0), page_size=ps, **table),
        "kv_fork": dict(pool=pool, src=i32(0), dst=i32(2), **table),
        "kv_compact": dict(pool=pool, tables=tables, refs=refs),
        "attn_forward": dict(ragged),
        "attn_backward": dict(do=do, o=o, lse=lse, **ragged),
    }


def in_order(name, kw):
    assert set(kw) <= set(NAMES[name])
    return [kw.get(a) for a in NAMES[name]]


def addresses():
    L = api.lib()
    return [ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in api._FAST_ENTRIES]


@pytest.fixture
def counted():
    """api._FAST with entry points that launch nothing and answer 7."""
    build.build()
    real = addresses()
    made = []
    # (the arguments are the caller's to clean up, so one that takes none stands for all)
    stand_in = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: made.append(1) or 7)
    at = ctypes.cast(stand_in, ctypes.c_void_p).value
    try:
        api._FAST.bind(tuple(a if n.endswith("_bytes") else at for n, a in zip(api._FAST_ENTRIES, real)))
        yield made
    finally:
        api._FAST.bind(tuple(real))


@pytest.mark.parametrize("name", NAMES)
def test_leaves_cpu_tensors(counted, name):
    fn = getattr(api._FAST, name)
    assert fn(*in_order(name, calls("cpu")[name])) is None
    assert fn(*[None] * len(NAMES[name])) is None
    assert fn(*[object()] * len(NAMES[name])) is None
    assert fn() is None
    assert not counted


def test_bind_refuses():
    build.build()
    api.lib()
    n = len(api._FAST_ENTRIES)
    for bad in (None, (), (1,) * (n - 1), (0,) * n, [1] * n):
        with pytest.raises(ValueError):
            api._FAST.bind(bad)
    with pytest.raises(TypeError):
        api._FAST.bind(("x",) * n)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_takes_the_plain_call(counted, name):
    kw = calls("cuda")[name]
    fn = getattr(api._FAST, name)
    assert fn(*in_order(name, kw)) == 7
    assert len(counted) == 1
    with pytest.raises(api.BitLinearError):
        getattr(api, "bl_" + name)(**kw)
    assert len(counted) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_leaves_what_is_wrong(counted, name):
    """Every tensor on the CPU, of another type, missing where it is needed, strided, and short."""
    fn = getattr(api._FAST, name)
    plain = calls("cuda")[name]
    for key, t in plain.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = [t.cpu(), t.to(torch.float64), t.to(torch.int64)]
        if t.dim() > 1:
            wrong.append(t.mT)
            wrong.append(t[..., ::2])
        if t.dim() == 1 and t.numel() > 1:
            wrong.append(t.repeat_interleave(2)[::2])
        if key in ("k", "v", "o", "lse", "do", "lengths", "k_pages", "v_pages", "active", "cu_k"):
            wrong.append(t[:-1].contiguous())
        if (key == "tables" and "lengths" in plain) or (key == "refs" and "pool" in plain):
            wrong.append(t[:-1].contiguous())
        if key == "pool":
            wrong.append(t[:, :-1].contiguous())
        if name == "rope_append" and key == "lengths":
            wrong.append(torch.cat([t, t]))
        for i, w in enumerate(wrong):
            assert fn(*in_order(name, {**plain, key: w})) is None, (name, key, i)
    for key in ("window", "sinks", "page_size", "max_q", "max_k"):
        if key in plain:
            assert fn(*in_order(name, {**plain, key: 1.0})) is None
            assert fn(*in_order(name, {**plain, key: 1 << 80})) is None
    for key, short in (("q_out", BF), ("k_out", BF), ("v_out", BF), ("out", F32), ("status", I32), ("n_live", I32),
                       ("dq", BF), ("dk", BF), ("dv", BF), ("workspace", torch.uint8)):
        if key in NAMES[name]:
            assert fn(*in_order(name, {**plain, key: torch.empty(0, dtype=short, device="cuda")})) is None, key
            assert fn(*in_order(name, {**plain, key: torch.empty(1 << 16, dtype=torch.float64, device="cuda")})) is None, key
    assert not counted


def run_both(name, monkeypatch, change=lambda kw: kw, taken=True):
    """The call's results and everything it was given, afterwards, by each way."""
    results = []
    for fast in (True, False):
        kw = change(calls("cuda")[name])
        with monkeypatch.context() as m:
            if fast:
                seen = []
                real = api._FAST

                class Spy:
                    def __getattr__(self, a):
                        def call(*args):
                            seen.append(getattr(real, a)(*args))
                            return seen[-1]
                        return call
                m.setattr(api, "_FAST", Spy())
            else:
                m.setattr(api, "_FAST", None)
            r = getattr(api, "bl_" + name)(**kw)
            if fast:
                assert len(seen) == 1 and (seen[0] is not None) == taken
        torch.cuda.synchronize()
        r = r if isinstance(r, tuple) else (r,)
        results.append(([x for x in r], {k: t for k, t in kw.items() if isinstance(t, torch.Tensor)}))
    (a, given_a), (b, given_b) = results
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and x.device == y.device
            assert torch.equal(x.cpu().view(torch.uint8), y.cpu().view(torch.uint8))
    for k in given_a:
        if k != "workspace":
            assert torch.equal(given_a[k].contiguous().cpu().view(torch.uint8),
                               given_b[k].contiguous().cpu().view(torch.uint8)), k


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_same_bits(name, monkeypatch):
    api.lib()
    run_both(name, monkeypatch)


def without(*keys):
    return lambda kw: {k: v for k, v in kw.items() if k not in keys}


def put(**new):
    return lambda kw: {**kw, **{k: v(kw) for k, v in new.items()}}


@pytest.mark.gpu
@pytest.mark.parametrize("name, change, taken", [
    ("rope_append", without("k_pages", "v_pages", "tables"), True),
    ("rope_append", without("k_pages", "v_pages", "tables", "lengths", "seq_ids", "keep_kv"), True),
    ("rope_append", without("k", "v", "k_pages", "v_pages", "tables", "out_dtype"), True),
    ("rope_append", without("q", "rope", "keep_kv"), True),
    ("rope_append", put(inverse=lambda kw: True, k_pages=lambda kw: None, v_pages=lambda kw: None), True),
    ("rope_append", put(keep_kv=lambda kw: 1), False),
    ("rope_append", put(k_out=lambda kw: torch.zeros(3, 2, 64, dtype=BF, device="cuda"), keep_kv=lambda kw: False), True),
    ("rope_append", put(q=lambda kw: torch.cat([kw["q"], kw["q"]], 1)[:, :4]), True),
    ("attn_decode", put(scale=lambda kw: None, return_lse=lambda kw: False, window=lambda kw: 5, sinks=lambda kw: 2), True),
    ("attn_decode", put(scale=lambda kw: 1), False),
    ("attn_decode", put(q=lambda kw: kw["q"].to(BF), seq_ids=lambda kw: None), True),
    ("attn_decode", put(q=lambda kw: kw["q"][:1], seq_ids=lambda kw: kw["seq_ids"][:1]), True),
    ("attn_decode", put(workspace=lambda kw: torch.empty(1 << 22, dtype=torch.uint8, device="cuda")), True),
    ("attn_decode", put(lse=lambda kw: torch.zeros(8, device="cuda"), return_lse=lambda kw: False), True),
    ("kv_extend", put(counts=lambda kw: kw["counts"] * 100), True),
    ("kv_fork", put(dst=lambda kw: kw["src"]), True),
    ("attn_forward", put(scale=lambda kw: 0.3, window=lambda kw: 0), True),
    ("attn_forward", put(o=lambda kw: torch.zeros(7, 4, 64, dtype=BF, device="cuda")), True),
    ("attn_backward", put(window=lambda kw: 0, do=lambda kw: torch.cat([kw["do"], kw["do"]], 1)[:, :4]), True),
])
def test_same_bits_of_other_calls(name, change, taken, monkeypatch):
    api.lib()
    run_both(name, monkeypatch, change, taken)


@pytest.mark.gpu
def test_stream_and_graph():
    """The launch and the allocations belong to the current stream, a captured one too."""
    api.lib()
    kw = calls("cuda")["attn_decode"]
    want = api.bl_attn_decode(**kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = api.bl_attn_decode(**kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = api.bl_attn_decode(**kw)
    held[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for pair in (got, held):
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
