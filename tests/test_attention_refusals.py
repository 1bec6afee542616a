"""The attention entry points without a GPU: the C ABI's checks of arguments
(host only, nothing is launched), the binding's checks of tensors, and the
formulas the GPU tests compare with, against differences."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api, build
from ternary_quantized_linear_bitlinear_b200.chain import DecodeChain
from ternary_quantized_linear_bitlinear_b200.kv import rope_table
from _attention import PageModel, attention, visible

OK, NULL, SHAPE, ALIGN, DTYPE, CUDA, TIMEOUT, WORKSPACE, DEVICE, INDEX = range(10)
A = 1 << 20  # a fake, 16-byte aligned "device address" (never dereferenced)
NO_GPU = (CUDA, DEVICE)


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake addresses must not reach a GPU")
    build.build()
    return api.lib()


def cache(k=A, v=A, tables=A, lengths=A, pages=64, ps=16, seqs=8, cols=10, dt=1):
    return ctypes.byref(api.KvCache(k, v, tables, lengths, pages, ps, seqs, cols, dt))


def test_status_string():
    build.build()
    assert api.status_string(INDEX).startswith("BL_ERR_INDEX")


def test_rope_append(L):
    def f(q=A, k=A, v=A, xdt=0, qs=768, ks=256, vs=256, T=4, Hq=12, Hkv=4, D=64, rope=A, rl=100, cu=None, B=4, ids=None,
          lens=None, ms=0, c=None, qo=A, ko=A, vo=A, odt=1):
        return L.bl_rope_append(q, k, v, xdt, qs, ks, vs, T, Hq, Hkv, D, rope, rl, 0, cu, B, ids, lens, ms, c, qo, ko, vo,
                                odt, None)
    assert f() in NO_GPU
    assert f(c=cache()) in NO_GPU
    assert f(q=None, qo=None) in NO_GPU
    assert f(k=None, v=None, ko=None, vo=None) in NO_GPU
    assert f(cu=A, B=2) in NO_GPU
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(k=None, v=None),
                dict(ko=None, vo=None), dict(q=None, k=None, v=None, qo=None, ko=None, vo=None),
                dict(k=None, v=None, ko=None, vo=None, c=cache()), dict(c=cache(k=None)), dict(c=cache(tables=None))):
        assert f(**bad) == NULL, bad
    assert f(xdt=2) == DTYPE and f(odt=5) == DTYPE and f(c=cache(dt=9)) == DTYPE
    for bad in (dict(D=24), dict(D=0), dict(D=144), dict(Hq=6), dict(Hkv=0), dict(T=0, B=0), dict(T=5), dict(qs=767),
                dict(ks=255), dict(rl=0), dict(B=0, cu=A), dict(c=cache(), lens=A, ms=8), dict(lens=A, ms=0),
                dict(c=cache(ps=12)), dict(c=cache(ps=4)), dict(c=cache(ps=2048)), dict(c=cache(pages=0)),
                dict(c=cache(seqs=0)), dict(c=cache(cols=1 << 28))):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(q=A + 4), dict(qs=769), dict(rope=A + 4), dict(qo=A + 8), dict(cu=A + 2), dict(c=cache(k=A + 8)),
                dict(vs=257)):
        assert f(**bad) == ALIGN, bad


def test_attn_decode(L):
    ws = L.bl_attn_decode_workspace_bytes(4, 12, 4, 64)
    assert ws > 0
    assert L.bl_attn_decode_workspace_bytes(0, 12, 4, 64) == 0
    assert L.bl_attn_decode_workspace_bytes(4, 12, 5, 64) == 0
    # eight heads a segment at most, whatever the group
    assert L.bl_attn_decode_workspace_bytes(4, 64, 1, 64) == L.bl_attn_decode_workspace_bytes(4, 8, 1, 64)

    def f(q=A, dt=0, qs=768, B=4, Hq=12, Hkv=4, D=64, c=cache(), ids=None, w=0, s=0, scale=0.125, wsp=A, wsb=ws, out=A,
          lse=None):
        return L.bl_attn_decode(q, dt, qs, B, Hq, Hkv, D, c, ids, w, s, scale, wsp, wsb, out, lse, None)
    assert f() in NO_GPU and f(lse=A, ids=A, w=5, s=1) in NO_GPU
    assert f(q=None) == NULL and f(c=None) == NULL and f(out=None) == NULL and f(c=cache(v=None)) == NULL
    assert f(dt=3) == DTYPE
    for bad in (dict(D=40), dict(Hq=13), dict(B=0), dict(B=9), dict(B=65536, ids=A), dict(w=-1), dict(s=-1), dict(qs=700),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)):
        assert f(**bad) == SHAPE, bad
    assert f(q=A + 8) == ALIGN and f(out=A + 4) == ALIGN and f(qs=770) == ALIGN and f(wsp=A + 8) == ALIGN
    assert f(wsp=None) == WORKSPACE and f(wsb=ws - 1) == WORKSPACE


def test_page_tables(L):
    def ext(t=A, ln=A, r=A, pages=64, ps=16, seqs=8, cols=10, ids=A, cnt=A, n=4, st=A, act=None):
        return L.bl_kv_extend(t, ln, r, pages, ps, seqs, cols, ids, cnt, n, st, act, None)
    assert ext() in NO_GPU and ext(act=A) in NO_GPU
    for bad in (dict(t=None), dict(ln=None), dict(r=None), dict(ids=None), dict(cnt=None), dict(st=None)):
        assert ext(**bad) == NULL
    for bad in (dict(n=0), dict(n=8193), dict(pages=0), dict(pages=(1 << 20) + 1), dict(ps=10), dict(seqs=0),
                dict(seqs=(1 << 17) + 1), dict(cols=0)):
        assert ext(**bad) == SHAPE, bad
    assert ext(ids=A + 1) == ALIGN and ext(act=A + 2) == ALIGN

    def free(t=A, ln=A, r=A, ids=A, n=4, ps=16):
        return L.bl_kv_free(t, ln, r, 64, ps, 8, 10, ids, n, None)
    assert free() in NO_GPU
    assert free(ids=None) == NULL and free(n=0) == SHAPE and free(ps=7) == SHAPE and free(r=A + 2) == ALIGN

    ws = L.bl_kv_fork_workspace_bytes(4)
    assert ws >= (1 + 3 * 4) * 4 and L.bl_kv_fork_workspace_bytes(0) == 0

    def fork(pool=A, planes=2, pb=1024, src=A, dst=A, n=4, wsp=A, wsb=ws, st=A):
        return L.bl_kv_fork(pool, planes, pb, A, A, A, 64, 16, 8, 10, src, dst, n, wsp, wsb, st, None)
    assert fork() in NO_GPU
    assert fork(pool=None) == NULL and fork(dst=None) == NULL and fork(st=None) == NULL
    assert fork(planes=0) == SHAPE and fork(pb=0) == SHAPE and fork(n=9000) == SHAPE
    assert fork(pb=1032) == ALIGN and fork(pool=A + 8) == ALIGN
    assert fork(wsp=None) == WORKSPACE and fork(wsb=ws - 1) == WORKSPACE

    wc = L.bl_kv_compact_workspace_bytes(64)
    assert wc >= (2 + 3 * 64) * 4 and L.bl_kv_compact_workspace_bytes(0) == 0

    def comp(pool=A, pages=64, pb=1024, wsb=wc, nl=A):
        return L.bl_kv_compact(pool, 2, pb, A, A, pages, 8, 10, A, wsb, nl, None)
    assert comp() in NO_GPU
    assert comp(pool=None) == NULL and comp(nl=None) == NULL and comp(pages=0) == SHAPE and comp(pb=24) == ALIGN
    assert comp(wsb=wc - 1) == WORKSPACE


def test_ragged(L):
    base = dict(qs=768, ks=256, vs=256, Tq=100, Tk=100, Hq=12, Hkv=4, D=64, cq=A, ck=A, B=2, mq=60, mk=60, w=0, s=0,
                scale=0.125)

    def fwd(q=A, k=A, v=A, o=A, lse=A, **kw):
        b = dict(base, **kw)
        return L.bl_attn_forward(q, k, v, *b.values(), o, lse, None)

    def bwd(do=A, q=A, k=A, v=A, o=A, lse=A, dos=768, wsp=A, wsb=None, dq=A, dk=A, dv=A, **kw):
        b = dict(base, **kw)
        if wsb is None:
            wsb = 1 << 30
        return L.bl_attn_backward(do, q, k, v, o, lse, dos, *b.values(), wsp, wsb, dq, dk, dv, None)

    for f in (fwd, bwd):
        assert f() in NO_GPU
        assert f(q=None) == NULL and f(lse=None) == NULL and f(cq=None) == NULL
        for bad in (dict(D=72), dict(Hkv=5), dict(Tq=0), dict(Tk=0), dict(B=0), dict(B=65536), dict(mq=0), dict(mk=1 << 24),
                    dict(w=-1), dict(s=-1), dict(scale=0.0), dict(scale=math.nan), dict(qs=767), dict(Tq=1 << 28)):
            assert f(**bad) == SHAPE, bad
        assert f(k=A + 8) == ALIGN and f(o=A + 8) == ALIGN and f(ck=A + 2) == ALIGN and f(vs=260) == ALIGN
    assert bwd(do=None) == NULL and bwd(dk=None) == NULL and bwd(dos=700) == SHAPE and bwd(dv=A + 8) == ALIGN
    need = L.bl_attn_backward_workspace_bytes(100, 100, 12, 4, 64, 2, 60, 60, 0, 0)
    assert need >= 100 * 12 * 4
    assert bwd(wsb=need - 1) == WORKSPACE and bwd(wsp=None) == WORKSPACE
    # sinks of a long batch add the pieces' sums
    more = L.bl_attn_backward_workspace_bytes(4000, 4000, 12, 4, 64, 2, 2000, 2000, 64, 4)
    assert more > L.bl_attn_backward_workspace_bytes(4000, 4000, 12, 4, 64, 2, 2000, 2000, 64, 0)
    assert L.bl_attn_backward_workspace_bytes(0, 1, 12, 4, 64, 1, 1, 1, 0, 0) == 0


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 4096
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = _FakeLib()
    monkeypatch.setattr(api, "lib", lambda: lib)
    monkeypatch.setattr(api, "_stream", lambda stream: 0)
    monkeypatch.setattr(api, "_is_cuda", lambda t: True)  # CPU tensors stand in for device buffers
    monkeypatch.setattr(api, "_device_index", lambda t: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    return lib


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_refuses_wrong_tensors(fake):
    x = torch.zeros(4, 6, 64)
    pages = torch.zeros(9, 2, 16, 64)
    tables, lengths = i32(5, 3), i32(5)
    api.bl_rope_append(x, x[:, :2], x[:, 2:4], torch.zeros(50, 64), None, lengths, None, pages, pages.clone(), tables)
    name, args = fake.calls[-1]
    assert name == "bl_rope_append" and args[4:7] == (384, 384, 384) and len(args[19]) == ctypes.sizeof(api.KvCache)
    bad = [
        (dict(q=x.half()), "float32 or bfloat16"),
        (dict(q=x[0]), "3-D"),
        (dict(q=x.transpose(1, 2)), "contiguous"),
        (dict(q=x, k=x[:, :2]), "together"),
        (dict(q=x, k=x[:3, :2], v=x[:3, :2]), "rows"),
        (dict(q=x, k=x[:, :2].bfloat16(), v=x[:, :2].bfloat16()), "must be torch.float32"),
        (dict(q=x, rope=torch.zeros(50, 32)), "rope"),
        (dict(q=x, out_dtype=torch.float16), "out_dtype"),
        (dict(q=x, q_out=torch.zeros(4, 6, 32)), "at least"),
        (dict(q=x, k=x, v=x, k_pages=pages), "together"),
        (dict(q=x, k=x[:, :2], v=x[:, :2], k_pages=pages, v_pages=pages), "tables"),
        (dict(q=x, k=x, v=x, k_pages=pages, v_pages=pages, tables=tables, lengths=lengths), "heads"),
        (dict(q=x, k=x[:, :2], v=x[:, :2], k_pages=pages, v_pages=pages, tables=tables, lengths=i32(4)), "elements"),
        (dict(q=x, lengths=i32(3)), "sequences"),
        (dict(q=x, seq_ids=i32(3)), "elements"),
        (dict(q=x, cu_seqlens=torch.zeros(3)), "int32"),
    ]
    n = len(fake.calls)
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            api.bl_rope_append(**kw)
    with pytest.raises(ValueError):
        api.bl_rope_append()
    q = x
    for call, match in (
        (lambda: api.bl_attn_decode(q, pages, pages, i32(3, 3), i32(3)), "batch entries"),
        (lambda: api.bl_attn_decode(q, pages[0], pages[0], tables, lengths), "4-D"),
        (lambda: api.bl_attn_decode(q, pages, pages.bfloat16(), tables, lengths), "v_pages"),
        (lambda: api.bl_attn_decode(q, pages, pages[:8], tables, lengths), "same shape"),
        (lambda: api.bl_attn_decode(q[..., :32].contiguous(), pages, pages, tables, lengths), "head size"),
        (lambda: api.bl_attn_decode(q, pages, pages, tables, lengths, out=torch.zeros(3)), "at least"),
        (lambda: api.bl_attn_decode(q, pages, pages, tables.long(), lengths), "int32"),
        (lambda: api.bl_kv_extend(tables, lengths, i32(9), i32(2), i32(3), 16), "counts"),
        (lambda: api.bl_kv_extend(tables, lengths, i32(3, 3), i32(2), i32(2), 16), "1-D"),
        (lambda: api.bl_kv_extend(tables, i32(4), i32(9), i32(2), i32(2), 16), "lengths"),
        (lambda: api.bl_kv_free(tables[0], lengths, i32(9), i32(2), 16), "2-D"),
        (lambda: api.bl_kv_fork(pages, tables, lengths, i32(8), i32(2), i32(2)), "number of pages"),
        (lambda: api.bl_kv_fork(pages, tables, lengths, i32(9), i32(2), i32(1)), "dst"),
        (lambda: api.bl_kv_compact(pages.half(), tables, i32(9)), "float32 or bfloat16"),
        (lambda: api.bl_attn_forward(x, x, x, i32(2), i32(2), 4, 4), "bfloat16"),
        (lambda: api.bl_attn_forward(*(x.bfloat16(),) * 3, i32(2), i32(3), 4, 4), "cu_k"),
        (lambda: api.bl_attn_forward(x.bfloat16(), x.bfloat16(), x[:, :3].bfloat16(), i32(2), i32(2), 4, 4), "heads"),
    ):
        with pytest.raises(ValueError, match=match):
            call()
    assert len(fake.calls) == n                  # none of them reached the library


def test_binding_on_cpu_tensors_without_a_stand_in():
    x = torch.zeros(4, 6, 64)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        api.bl_rope_append(x)


def test_chain_refuses_a_cache_that_does_not_fit(monkeypatch):
    class C:
        pool, head_dim, kv_heads, page_size = torch.zeros(2, 2, 4, 4, 8, 64), 64, 4, 8
        tables = i32(3, 5)

    chain = DecodeChain.__new__(DecodeChain)
    chain.M, chain.cache = 2, C()
    lay = dict(k=(None, None, 256, 768))
    chain._check_cache([lay, lay], 768, i32(2), torch.zeros(40, 64))
    for layers, hidden, ids, rope, match in (([lay], 768, i32(2), None, "layers"), ([lay, lay], 700, i32(2), None, "heads"),
                                             ([dict(k=(None, None, 128, 768))] * 2, 768, i32(2), None, "heads"),
                                             ([lay, lay], 768, i32(3), None, "seq_ids"), ([lay, lay], 768, None, None, "seq_ids"),
                                             ([lay, lay], 768, i32(2), torch.zeros(39, 64), "rope")):
        with pytest.raises(ValueError, match=match):
            chain._check_cache(layers, hidden, ids, rope)


def test_rope_table_is_the_angles():
    t = rope_table(5000, 8, theta=100.0, device="cpu")
    for p in (0, 1, 4999):
        for i in range(4):
            a = p * 100.0 ** (-2 * i / 8)
            assert abs(t[p, i].item() - math.cos(a)) < 2.0 ** -24
            assert abs(t[p, 4 + i].item() - math.sin(a)) < 2.0 ** -24


def test_gradient_formulas_against_differences():
    """The formulas the GPU's gradients are compared with, at random directions
    of every input: the central difference of sum(o * do) over a step e is the
    directional derivative within e^2 of a third derivative."""
    g = torch.Generator().manual_seed(2)
    n, m, D, scale = 7, 9, 16, 0.3
    q, do = (torch.randn(n, D, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(m, D, generator=g, dtype=torch.float64) for _ in range(2))
    for window, sinks in ((0, 0), (3, 1), (1, 0)):
        see = visible(n, m, window, sinks)
        o, _, P = attention(q, k, v, see, scale)
        dS = P * (do @ v.T - (do * o).sum(1, keepdim=True))
        grads = {"q": scale * dS @ k, "k": scale * dS.T @ q, "v": P.T @ do}
        for name, x in (("q", q), ("k", k), ("v", v)):
            r = torch.randn(x.shape, generator=g, dtype=torch.float64)
            e = 1e-5
            at = []
            for sign in (1, -1):
                a = dict(q=q, k=k, v=v)
                a[name] = x + sign * e * r
                at.append((attention(a["q"], a["k"], a["v"], see, scale)[0] * do).sum().item())
            assert abs((at[0] - at[1]) / (2 * e) - (grads[name] * r).sum().item()) < 1e-7


def test_page_model_on_a_hand_example():
    m = PageModel(6, 8, 3, 3)
    assert m.extend([0, 1], [9, 3]) == 0 and m.tables[0] == [0, 1, -1] and m.tables[1] == [2, -1, -1]
    assert m.fork([0], [2]) == 0 and m.tables[2] == [0, 3, -1] and m.moves == [(1, 3)] and m.refs == [2, 1, 1, 1, 0, 0]
    m.free([0])
    assert m.refs == [1, 0, 1, 1, 0, 0] and m.lengths == [0, 3, 9]
    assert m.compact() == 3 and m.moves == [(3, 1)] and m.tables[2] == [0, 1, -1] and m.refs == [1, 1, 1, 0, 0, 0]
