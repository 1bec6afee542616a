"""The attention operators of the library and the cases they are measured at.

Four operators, those between the q, k, v projections of a decoder layer and
its o projection:

  append   rotary positions on q and k, and the new K/V rows into the pages
           of a cache (api.bl_rope_append)
  decode   attention of one new token per sequence over the paged cache
           (api.bl_attn_decode)
  pages    sequences of the cache admitted, forked, freed; the pool compacted
           (api.bl_kv_extend, bl_kv_fork, bl_kv_free, bl_kv_compact)
  forward, train
           causal attention over a ragged batch with a sliding window and
           first tokens that stay visible, and its gradients
           (api.bl_attn_forward, api.bl_attn_backward)

With own = False `run` computes them from elementary torch operations in
float32, with own = True through the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's writes: 8 sequences of the 125M student, f32 projections
        dict(name="append-8", op="append", B=8, ragged=False, new=1, past=1500, Hq=12, Hkv=4, D=64, ps=16,
             src="f32", out="f32", cache="bf16", rope=True, mix=1),
        # a prompt of 8192 tokens in five requests through one 1.4B layer, rounded for the prefill attention
        dict(name="append-8192", op="append", B=5, ragged=True, new=3500, past=0, Hq=12, Hkv=4, D=128, ps=64,
             src="f32", out="bf16", cache="bf16", rope=True, mix=2),
        # a single chat of a few hundred tokens with the 125M student: latency
        dict(name="decode-1x701", op="decode", B=1, ragged=False, len=701, Hq=12, Hkv=4, D=64, ps=16, src="f32",
             cache="bf16", window=0, sinks=0, mix=3),
        # a full batch of very different lengths on the 4B shape (20 heads, not shared), windowed with sinks
        dict(name="decode-64-window", op="decode", B=64, ragged=True, len=16384, Hq=20, Hkv=20, D=128, ps=32,
             src="f32", cache="bf16", window=1024, sinks=4, mix=4),
        # long contexts of the 1.4B shape: the cache's bytes decide
        dict(name="decode-8x65000", op="decode", B=8, ragged=False, len=65000, Hq=12, Hkv=4, D=128, ps=64,
             src="bf16", cache="bf16", window=0, sinks=0, mix=5),
        # four samples forked from one prompt of the 125M student, one request finished and one admitted
        dict(name="turnover-4", op="turnover", planes=24, pages=256, Hkv=4, D=64, ps=16, cache="bf16", seqs=16, cols=32,
             live=6, len=300, ragged=True, forks=4, mix=6),
        # a busy server of the 1.4B shape, 24 layers: 64 samples forked, 64 requests replaced
        dict(name="turnover-64", op="turnover", planes=48, pages=4000, Hkv=4, D=128, ps=32, cache="bf16", seqs=256,
             cols=64, live=128, len=1500, ragged=True, forks=64, mix=7),
        # the pool after half of its requests ended, moved together
        dict(name="compact-4000", op="compact", planes=48, pages=4000, Hkv=4, D=128, ps=32, cache="bf16", seqs=128,
             cols=64, live=100, len=1500, ragged=True, forks=0, mix=8),
        # prefill of three short prompts with the 125M student
        dict(name="forward-3x201", op="forward", B=3, ragged=True, q=201, past=0, Hq=12, Hkv=4, D=64, window=0, sinks=0,
             mix=9),
        # prefill of 8192 tokens through a 1.4B layer, sliding window 1024, four sinks
        dict(name="forward-8192-window", op="forward", B=1, ragged=False, q=8192, past=0, Hq=12, Hkv=4, D=128,
             window=1024, sinks=4, mix=10),
        # a training step of the 125M student on sequences of odd lengths, windowed
        dict(name="train-6x1000", op="train", B=6, ragged=True, q=1000, past=0, Hq=12, Hkv=4, D=64, window=256, sinks=1,
             mix=11),
        # the 4B layer's training batch, 16 sequences of 2048
        dict(name="train-16x2048", op="train", B=16, ragged=False, q=2048, past=0, Hq=20, Hkv=20, D=128, window=0,
             sinks=0, mix=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "turnover", "compact", "forward", "train"])
    heads = rng.choice([(12, 4), (12, 4), (20, 20), (8, 1), (25, 25), (6, 2)])
    D = rng.choice([64, 64, 128, 128, 32, 80, 96])
    c = dict(op=op, Hq=heads[0], Hkv=heads[1], D=D, mix=rng.randrange(1 << 30), ragged=rng.random() < 0.7)
    if op == "append":
        c.update(B=_spread(rng, 1, 32), ps=rng.choice([16, 32, 64, 128]), src=rng.choice(["f32", "bf16"]),
                 out=rng.choice(["f32", "bf16"]), cache=rng.choice(["bf16", "bf16", "f32"]), rope=rng.random() < 0.8)
        if rng.random() < 0.5:
            c.update(B=_spread(rng, 1, 128), new=1, ragged=False, past=_spread(rng, 1, 8000))
        else:
            c.update(new=max(1, _spread(rng, 16, 8192) // c["B"]), past=rng.choice([0, 0, 777]))
    elif op == "decode":
        c.update(B=_spread(rng, 1, 128), ps=rng.choice([8, 16, 32, 64, 128]), src=rng.choice(["f32", "f32", "bf16"]),
                 cache=rng.choice(["bf16", "bf16", "bf16", "f32"]), window=rng.choice([0, 0, 1024, 1000]))
        c["sinks"] = rng.choice([0, 1, 4, 37]) if c["window"] else 0
        c["len"] = _spread(rng, 20, max(40, 130_000_000 // (c["B"] * heads[1] * D) // 2))
    elif op in ("turnover", "compact"):
        c.update(Hq=0, planes=2 * rng.choice([1, 12, 24]), ps=rng.choice([16, 32, 64]), cache=rng.choice(["bf16", "f32"]),
                 len=_spread(rng, 30, 1400), live=_spread(rng, 4, 100), forks=_spread(rng, 1, 48))
        c["D"], c["Hkv"] = rng.choice([64, 128]), rng.choice([1, 4])
        c["seqs"] = c["live"] + 2 * c["forks"] + 4
        c["cols"] = 2 + (c["len"] + c["ps"] - 1) // c["ps"]
        if op == "compact":
            c["forks"] = 0
        # room for every sequence at its longest, bounded so that the pool stays below 1.6 GB
        c["pages"] = 16 + (c["live"] + c["forks"]) * c["cols"]
        c["planes"] = max(1, min(c["planes"], 1_600_000_000 // (c["pages"] * c["Hkv"] * c["ps"] * c["D"] * 4)))
    else:
        c.update(B=_spread(rng, 1, 16), window=rng.choice([0, 0, 256, 1024, 100]))
        c["sinks"] = rng.choice([0, 1, 4, 40]) if c["window"] else 0
        c["past"] = rng.choice([0, 0, 333]) if op == "forward" else 0
        most = int(math.sqrt(600_000_000 / (c["B"] * heads[0]))) - c["past"]
        c["q"] = _spread(rng, 16, max(32, min(8000, most)))
    return c


# ---------------------------------------------------------------------------
# inputs

def _lens(case, n, most, least=1):
    """n lengths of at most `most`, the first of them `most`, from the case alone."""
    if not case["ragged"]:
        return [most] * n
    rng = random.Random(case["mix"])
    return [most] + [_spread(rng, max(1, min(least, most)), most) for _ in range(n - 1)]


def _table(rows, cols, pages, order, dev):
    """Rows of page numbers, taken in the given order, -1 behind them."""
    t = torch.full((len(rows), cols), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(rows):
        t[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    assert at <= pages
    return t.to(dev)


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _append_lens(case):
    new = _lens(case, case["B"], case["new"], 1 + case["new"] // 20)
    past = _lens(dict(case, mix=case["mix"] + 1, ragged=True), case["B"], case["past"]) if case["past"] else [0] * case["B"]
    return new, past


def _attn_lens(case):
    q = _lens(case, case["B"], case["q"], 1 + case["q"] // 8)
    return q, [n + case["past"] for n in q]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    op = case["op"]
    s = dict(case=case, op=op)
    rng = random.Random(seed * 7919 + 13)
    if op == "append":
        new, past = _append_lens(case)
        T, H, Hk, D, ps = sum(new), case["Hq"], case["Hkv"], case["D"], case["ps"]
        need = [-(-(a + b) // ps) for a, b in zip(new, past)]
        pages = sum(need) + 3
        order = list(range(pages))
        rng.shuffle(order)
        # q, k and v are the columns of one projection output
        qkv = normal(T, H + 2 * Hk, D, dtype=_T[case["src"]])
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], cu=_i32(_cum(new), dev),
                 lengths=_i32([a + b for a, b in zip(new, past)], dev), tables=_table(need, max(need), pages, order, dev),
                 k_pages=normal(pages, Hk, ps, D, dtype=_T[case["cache"]]),
                 v_pages=normal(pages, Hk, ps, D, dtype=_T[case["cache"]]))
        if case["rope"]:
            n = max(a + b for a, b in zip(new, past))
            inv = 1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
            ang = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv[None]
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            s["rope"] = None
    elif op == "decode":
        B, H, Hk, D, ps = case["B"], case["Hq"], case["Hkv"], case["D"], case["ps"]
        lens = _lens(case, B, case["len"])
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 2
        order = list(range(pages))
        rng.shuffle(order)
        s.update(q=normal(B, H, D, dtype=_T[case["src"]], std=1.5), lengths=_i32(lens, dev),
                 tables=_table(need, max(need), pages, order, dev),
                 k_pages=normal(pages, Hk, ps, D, dtype=_T[case["cache"]]),
                 v_pages=normal(pages, Hk, ps, D, dtype=_T[case["cache"]]))
    elif op in ("turnover", "compact"):
        pages, ps, cols, nseq, live = case["pages"], case["ps"], case["cols"], case["seqs"], case["live"]
        lens = _lens(case, live, case["len"], 1 + case["len"] // 10)
        need = [-(-n // ps) for n in lens]
        order = list(range(pages))
        rng.shuffle(order)
        tables = torch.full((nseq, cols), -1, dtype=torch.int32, device=dev)
        tables[:live] = _table(need, cols, pages, order, dev)
        lengths = torch.zeros(nseq, dtype=torch.int32, device=dev)
        lengths[:live] = _i32(lens, dev)
        refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        refs[torch.tensor(order[:sum(need)], device=dev)] = 1
        pool = normal(case["planes"], pages, case["Hkv"], ps, case["D"], dtype=_T[case["cache"]])
        s.update(pool=pool, tables=tables, lengths=lengths, refs=refs)
        if op == "turnover":
            k = case["forks"]
            gone = list(range(live))
            rng.shuffle(gone)
            gone = gone[:min(k, live // 2)]
            kept = [i for i in range(live) if i not in gone]
            s.update(src=_i32([kept[i % max(1, len(kept) // 2)] for i in range(k)], dev),
                     dst=_i32(list(range(live, live + k)), dev), admit=_i32(gone, dev),
                     counts=_i32([1 + rng.randrange(case["len"]) for _ in gone], dev),
                     gone=_i32(gone + list(range(live, live + k)), dev),
                     status=torch.zeros(1, dtype=torch.int32, device=dev))
        else:
            s.update(tables0=tables.clone(), refs0=refs.clone(), n_live=torch.zeros(1, dtype=torch.int32, device=dev))
    else:
        nq, nk = _attn_lens(case)
        H, Hk, D = case["Hq"], case["Hkv"], case["D"]
        s.update(q=normal(sum(nq), H, D, dtype=torch.bfloat16), k=normal(sum(nk), Hk, D, dtype=torch.bfloat16),
                 v=normal(sum(nk), Hk, D, dtype=torch.bfloat16), cu_q=_i32(_cum(nq), dev), cu_k=_i32(_cum(nk), dev),
                 most_q=max(nq), most_k=max(nk))
        if op == "train":
            s["do"] = normal(sum(nq), H, D, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return _own(s)
    return {"append": _append, "decode": _decode, "turnover": _turnover, "compact": _compact, "forward": _forward,
            "train": _train}[s["op"]](s)


def _own(s):
    from ternary_quantized_linear_bitlinear_b200 import api

    c, op = s["case"], s["op"]
    if op == "append":
        q, _, _ = api.bl_rope_append(s["q"], s["k"], s["v"], rope=s["rope"], cu_seqlens=s["cu"], lengths=s["lengths"],
                                     k_pages=s["k_pages"], v_pages=s["v_pages"], tables=s["tables"],
                                     out_dtype=_T[c["out"]])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "decode":
        o, lse = api.bl_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["lengths"], window=c["window"],
                                    sinks=c["sinks"], return_lse=True)
        return {"o": o, "lse": lse}
    if op == "turnover":
        api.bl_kv_free(s["tables"], s["lengths"], s["refs"], s["gone"], c["ps"])
        api.bl_kv_extend(s["tables"], s["lengths"], s["refs"], s["admit"], s["counts"], c["ps"], status=s["status"])
        api.bl_kv_fork(s["pool"], s["tables"], s["lengths"], s["refs"], s["src"], s["dst"], status=s["status"])
        return {k: s[k] for k in ("pool", "tables", "lengths", "refs", "status")}
    if op == "compact":
        # the page numbers of the scattered pool, so that every pass moves the same pages
        s["tables"].copy_(s["tables0"])
        s["refs"].copy_(s["refs0"])
        api.bl_kv_compact(s["pool"], s["tables"], s["refs"], n_live=s["n_live"])
        return {k: s[k] for k in ("pool", "tables", "refs", "n_live")}
    o, lse = api.bl_attn_forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["most_q"], s["most_k"],
                                 window=c["window"], sinks=c["sinks"])
    if op == "forward":
        return {"o": o, "lse": lse}
    dq, dk, dv = api.bl_attn_backward(s["do"], s["q"], s["k"], s["v"], o, lse, s["cu_q"], s["cu_k"], s["most_q"],
                                      s["most_k"], window=c["window"], sinks=c["sinks"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# the plain forms

def _append(s):
    c = s["case"]
    cu, T, D = s["cu"].long(), s["q"].shape[0], c["D"]
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lengths"].long()[b] - cu[b + 1] + t

    def turn(x):
        x = x.float()
        if s["rope"] is None:
            return x
        cos, sin = s["rope"][pos][:, None].split(D // 2, -1)
        lo, hi = x.split(D // 2, -1)
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)

    page, slot = s["tables"].long()[b, pos // c["ps"]], pos % c["ps"]
    s["k_pages"][page, :, slot] = turn(s["k"]).to(s["k_pages"].dtype)
    s["v_pages"][page, :, slot] = s["v"].to(s["v_pages"].dtype)
    return {"q": turn(s["q"]).to(_T[c["out"]]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _decode(s):
    c = s["case"]
    B, H, D = s["q"].shape
    lens = s["lengths"].long()
    table = s["tables"].long().clamp(min=0)
    # [B, Hkv, keys, D]
    k = s["k_pages"][table].transpose(1, 2).flatten(2, 3).float()
    v = s["v_pages"][table].transpose(1, 2).flatten(2, 3).float()
    j = torch.arange(k.shape[2], device=k.device)[None]
    seen = j < lens[:, None]
    if c["window"]:
        seen = seen & ((j >= lens[:, None] - c["window"]) | (j < c["sinks"]))
    q = s["q"].float().view(B, c["Hkv"], -1, D)
    x = (q @ k.transpose(2, 3)) / math.sqrt(D)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / z
    return {"o": o.view(B, H, D).to(s["q"].dtype), "lse": (m + torch.log(z)).view(B, H)}


def _release(s, ids):
    c = s["case"]
    rows = s["tables"][ids]
    used = torch.arange(rows.shape[1], device=rows.device)[None] < -(-s["lengths"][ids] // c["ps"])[:, None]
    s["refs"].index_add_(0, rows[used].long(), torch.full_like(rows[used], -1))
    s["tables"][ids] = -1
    s["lengths"][ids] = 0


def _admit(s, ids, counts):
    ps = s["case"]["ps"]
    have, want = -(-s["lengths"][ids] // ps), -(-(s["lengths"][ids] + counts) // ps)
    rows = s["tables"][ids]
    col = torch.arange(rows.shape[1], device=rows.device)[None]
    put = (col >= have[:, None]) & (col < want[:, None])
    pages = torch.nonzero(s["refs"] == 0).flatten()[:int(put.sum())]
    rows[put] = pages.int()
    s["tables"][ids] = rows
    s["refs"][pages] = 1
    s["lengths"][ids] += counts


def _turnover(s):
    ps = s["case"]["ps"]
    _release(s, s["gone"].long())
    _admit(s, s["admit"].long(), s["counts"])
    src, dst = s["src"].long(), s["dst"].long()
    n = s["lengths"][src]
    full = (n // ps).long()
    rows = s["tables"][src]
    shared = torch.arange(rows.shape[1], device=rows.device)[None] < full[:, None]
    s["refs"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    part = torch.nonzero(n % ps).flatten()
    old = rows[part, full[part]].long()
    new = torch.nonzero(s["refs"] == 0).flatten()[:part.numel()]
    rows[part, full[part]] = new.int()
    s["refs"][new] = 1
    s["pool"][:, new] = s["pool"][:, old]
    s["tables"][dst] = rows
    s["lengths"][dst] = n
    s["status"].zero_()
    return {k: s[k] for k in ("pool", "tables", "lengths", "refs", "status")}


def _compact(s):
    s["tables"].copy_(s["tables0"])
    s["refs"].copy_(s["refs0"])
    refs, tables = s["refs"], s["tables"]
    n = int((refs > 0).sum())
    holes = torch.nonzero(refs[:n] == 0).flatten()
    movers = torch.nonzero(refs[n:] > 0).flatten() + n
    s["pool"][:, holes] = s["pool"][:, movers]
    to = torch.arange(refs.numel(), device=refs.device, dtype=torch.int32)
    to[movers] = holes.int()
    tables.copy_(torch.where(tables >= 0, to[tables.long().clamp(min=0)], tables))
    refs[holes] = refs[movers]
    refs[movers] = 0
    s["n_live"].fill_(n)
    return {k: s[k] for k in ("pool", "tables", "refs", "n_live")}


def _padded(s):
    """The ragged batch as [B, most, ...] with the rows' places and what each query sees."""
    c = s["case"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(s["most_q"], device=cq.device), torch.arange(s["most_k"], device=cq.device)
    nq, nk = (cq[1:] - cq[:-1])[:, None], (ck[1:] - ck[:-1])[:, None]
    at_q, at_k = i[None] < nq, j[None] < nk
    pos = (nk - nq + i[None])[:, :, None]
    seen = at_q[:, :, None] & at_k[:, None] & (j[None, None] <= pos)
    if c["window"]:
        seen = seen & ((pos - j[None, None] < c["window"]) | (j[None, None] < c["sinks"]))

    def pad(x, at):
        out = torch.zeros(*at.shape, *x.shape[1:], device=x.device)
        out[at] = x.float()
        return out

    q, k, v = pad(s["q"], at_q), pad(s["k"], at_k), pad(s["v"], at_k)
    group = c["Hq"] // c["Hkv"]
    q = q.unflatten(2, (c["Hkv"], group)).permute(0, 2, 3, 1, 4)
    return q, k.permute(0, 2, 1, 3)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None], seen[:, None, None], at_q, at_k, pad


def _soft(q, k, v, seen):
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True).clamp(min=1e-30)
    p = p.div_(z)
    return p, p @ v, (m + torch.log(z)).squeeze(-1)


def _rows(x, at):
    """[B, Hkv, group, most, D] -> [T, H, D]."""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3)[at]


def _forward(s):
    q, k, v, seen, at_q, _, _ = _padded(s)
    _, o, lse = _soft(q, k, v, seen)
    return {"o": _rows(o, at_q).bfloat16(), "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[at_q].t().contiguous()}


def _train(s):
    q, k, v, seen, at_q, at_k, pad = _padded(s)
    c = s["case"]
    p, o, lse = _soft(q, k, v, seen)
    do = pad(s["do"], at_q).unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    scale = 1.0 / math.sqrt(c["D"])
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    return {"o": _rows(o, at_q).bfloat16(), "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[at_q].t().contiguous(),
            "dq": _rows(dq, at_q).bfloat16(), "dk": dk.permute(0, 2, 1, 3)[at_k].bfloat16(),
            "dv": dv.permute(0, 2, 1, 3)[at_k].bfloat16()}


# ---------------------------------------------------------------------------
# what a pass cannot do without

_SIZE = {"f32": 4, "bf16": 2}


def _pairs(nq, nk, window, sinks):
    """Visible (query, key) pairs of one sequence and head."""
    total = 0
    for i in range(nq):
        pos = nk - nq + i
        if pos < 0:
            continue
        n = pos + 1
        if window and n > window:
            n = window + min(sinks, n - window)
        total += n
    return total


def work(case):
    op = case["op"]
    if op == "append":
        new, past = _append_lens(case)
        T = sum(new)
        b = T * case["D"] * ((case["Hq"] + 2 * case["Hkv"]) * _SIZE[case["src"]] + case["Hq"] * _SIZE[case["out"]]
                             + 2 * case["Hkv"] * _SIZE[case["cache"]])
        if case["rope"]:
            b += max(new) * case["D"] * 4
        return {"bytes": b, "flops": 3 * T * case["D"] * (case["Hq"] + case["Hkv"]) if case["rope"] else 0}
    if op == "decode":
        keys = sum(min(n, case["window"] + min(case["sinks"], max(0, n - case["window"]))) if case["window"] else n
                   for n in _lens(case, case["B"], case["len"]))
        return {"bytes": keys * case["Hkv"] * case["D"] * 2 * _SIZE[case["cache"]]
                + case["B"] * case["Hq"] * (2 * case["D"] * _SIZE[case["src"]] + 4),
                "flops": 4 * keys * case["Hq"] * case["D"]}
    if op in ("turnover", "compact"):
        page = case["planes"] * case["Hkv"] * case["ps"] * case["D"] * _SIZE[case["cache"]]
        lens = _lens(case, case["live"], case["len"], 1 + case["len"] // 10)
        used = sum(-(-n // case["ps"]) for n in lens)
        moved = case["forks"] if op == "turnover" else int(used * (1 - used / case["pages"]))
        return {"bytes": 2 * moved * page + 4 * (case["pages"] + case["seqs"] * case["cols"]), "flops": 0}
    nq, nk = _attn_lens(case)
    H, Hk, D = case["Hq"], case["Hkv"], case["D"]
    pairs = sum(_pairs(a, b, case["window"], case["sinks"]) for a, b in zip(nq, nk))
    b = (sum(nq) * 2 * H + sum(nk) * 2 * Hk) * D * 2 + sum(nq) * H * 4
    f = 4 * pairs * H * D
    if op == "train":
        b += (sum(nq) * 2 * H + sum(nk) * 2 * Hk) * D * 2
        f += 10 * pairs * H * D
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "turnover": _exact_turnover, "compact": _exact_compact,
            "forward": _exact_attn, "train": _exact_attn}[case["op"]](case, s)


def _exact_append(c, s):
    """Token by token: page and slot from the position, rotation as a product of complex numbers."""
    new, past = _append_lens(c)
    D, ps = c["D"], c["ps"]
    where = [(b, past[b] + i) for b in range(c["B"]) for i in range(new[b])]
    table = s["tables"].cpu().tolist()
    page = torch.tensor([table[b][p // ps] for b, p in where], device="cuda")
    slot = torch.tensor([p % ps for _, p in where], device="cuda")
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if s["rope"] is not None:
        r = s["rope"].double()[torch.tensor([p for _, p in where], device="cuda")]
        w = torch.complex(r[:, :D // 2], r[:, D // 2:])[:, None]

        def turn(x):
            z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * w
            return torch.cat([z.real, z.imag], -1)
        q, k = turn(q), turn(k)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    kp[page, :, slot] = k
    vp[page, :, slot] = v
    return {"q": q, "k_pages": kp, "v_pages": vp}


def _exact_decode(c, s):
    B, H, D, ps = c["B"], c["Hq"], c["D"], c["ps"]
    o = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lengths"].cpu().tolist()
    for b in range(B):
        n = lens[b]
        keys = [j for j in range(n) if not c["window"] or j >= n - c["window"] or j < c["sinks"]]
        if not keys:
            continue
        j = torch.tensor(keys, device="cuda")
        page = s["tables"][b].long()[j // ps]
        k, v = s["k_pages"][page, :, j % ps].double(), s["v_pages"][page, :, j % ps].double()
        for h in range(H):
            x = k[:, h * c["Hkv"] // H] @ s["q"][b, h].double() * D ** -0.5
            lse[b, h] = torch.logsumexp(x, 0)
            o[b, h] = torch.softmax(x, 0) @ v[:, h * c["Hkv"] // H]
    return {"o": o, "lse": lse}


def _exact_turnover(c, s):
    """The same bookkeeping on lists, one sequence after the other."""
    ps = c["ps"]
    tables, lens, refs = s["tables"].cpu().tolist(), s["lengths"].cpu().tolist(), s["refs"].cpu().tolist()

    def take():
        p = refs.index(0)
        refs[p] = 1
        return p

    for q in s["gone"].cpu().tolist():
        for j in range(-(-lens[q] // ps)):
            refs[tables[q][j]] -= 1
            tables[q][j] = -1
        lens[q] = 0
    for q, n in zip(s["admit"].cpu().tolist(), s["counts"].cpu().tolist()):
        for j in range(-(-lens[q] // ps), -(-(lens[q] + n) // ps)):
            tables[q][j] = take()
        lens[q] += n
    moves = []
    for a, b in zip(s["src"].cpu().tolist(), s["dst"].cpu().tolist()):
        for j in range(-(-lens[a] // ps)):
            if (j + 1) * ps <= lens[a]:
                refs[tables[a][j]] += 1
                tables[b][j] = tables[a][j]
            else:
                tables[b][j] = take()
                moves.append((tables[a][j], tables[b][j]))
        lens[b] = lens[a]
    pool = s["pool"].clone()
    for a, b in moves:
        pool[:, b] = pool[:, a]
    return {"pool": pool, "tables": _i32(tables, "cuda"), "lengths": _i32(lens, "cuda"), "refs": _i32(refs, "cuda"),
            "status": _i32([0], "cuda")}


def _exact_compact(c, s):
    tables, refs = s["tables0"].cpu().tolist(), s["refs0"].cpu().tolist()
    pool, moved = s["pool"].clone(), {}
    n = sum(r > 0 for r in refs)
    holes = iter([p for p in range(n) if refs[p] == 0])
    for p in range(n, len(refs)):
        if refs[p] > 0:
            h = next(holes)
            pool[:, h] = pool[:, p]
            moved[p], refs[h], refs[p] = h, refs[p], 0
    return {"pool": pool, "tables": _i32([[moved.get(p, p) for p in row] for row in tables], "cuda"),
            "refs": _i32(refs, "cuda"), "n_live": _i32([n], "cuda")}


def _exact_attn(c, s):
    """Sequence by sequence and head by head, the gradients by differentiating the definition."""
    train = c["op"] == "train"
    nq, nk = _attn_lens(c)
    cq, ck = _cum(nq), _cum(nk)
    H, Hk, D = c["Hq"], c["Hkv"], c["D"]
    q, k, v = (s[n].double().requires_grad_(train) for n in "qkv")
    o = torch.zeros(cq[-1], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((H, cq[-1]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        i = torch.arange(nk[b] - nq[b], nk[b], device="cuda")[:, None]
        j = torch.arange(nk[b], device="cuda")[None]
        hidden = (j > i) | ((i - j >= c["window"]) & (j >= c["sinks"])) if c["window"] else j > i
        for h in range(H):
            kh, vh = k[ck[b]:ck[b + 1], h // (H // Hk)], v[ck[b]:ck[b + 1], h // (H // Hk)]
            x = torch.where(hidden, -math.inf, q[cq[b]:cq[b + 1], h] @ kh.t() * D ** -0.5)
            lse[h, cq[b]:cq[b + 1]] = torch.logsumexp(x.detach(), 1)
            out = torch.softmax(x, 1) @ vh
            o[cq[b]:cq[b + 1], h] = out.detach()
            if train:
                out.backward(s["do"][cq[b]:cq[b + 1], h].double())
    if not train:
        return {"o": o, "lse": lse}
    return {"o": o, "lse": lse, "dq": q.grad, "dk": k.grad, "dv": v.grad}
