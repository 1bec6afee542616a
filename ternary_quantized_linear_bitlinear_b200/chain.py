"""A dependency-ordered decode step through a stack of BitLinear layers.

Each layer feeds the next, as one token step of a decoder does, with every
projection a BitLinear of this library and nothing computed outside it:

    Y_q, Y_k, Y_v = BitLinear_{q,k,v}(x)           one fused decode launch
    Y_o           = BitLinear_o(SubLN(Y_q))        one fused decode launch
    Y_g, Y_u      = BitLinear_{gate,up}(Y_o)       one fused decode launch
    x_q, s        = quant(SubLN(relu(Y_g)^2 Y_u))  bl_ffn_act_quant
    x'            = BitLinear_down(x_q, s)         one decode launch
    (x' is the next layer's x)

Without a cache the o projection reads the q projection's output in the
attention's place (same width).  With one (kv.PagedKV) each token is the next
of its own sequence, and between the two stands the attention:

    the sequences grow by one token                bl_kv_extend, once per step
    q' = rope(Y_q); rope(Y_k), Y_v -> pages        bl_rope_append
    A = attention(q', pages)                       bl_attn_decode (two launches)
    Y_o = BitLinear_o(SubLN(A))

SubLN sits before o_proj and down_proj ("BitDistill", Stage 1 -- Architectural refinement with SubLN),
ReLU^2 gates the FFN ("SLM750-Edge", Key Architectural Features).  The
weights are static, so every projection launch is a programmatic dependent
of the launch before it (BL_FWD_WEIGHTS_READY): it streams its weights while
that launch finishes, and reads its activations only after.

This module only arranges buffers and calls the library's entry points.
"""
from __future__ import annotations

import torch

from . import api

# projection order inside a layer, and the launch groups of one layer
PROJ = ("q", "k", "v", "o", "gate", "up", "down")


class DecodeChain:
    """layers: list of dicts name -> (packed uint8 [N, K/4], gamma float32 [1],
    N, K) for the seven projections; gains: list of (g_o [hidden],
    g_down [ffn]) float32 device tensors.  M tokens per step (M <= 16).
    With record=True every projection also writes its x_q, s and int32
    accumulators (for checking), else only Y.

    cache: a kv.PagedKV with a layer per entry of `layers`; seq_ids int32 [M]
    (device) the sequences of the M tokens, negative for a padded one (read by
    every step: write new ids into it between steps); rope float32 [positions,
    head_dim] (kv.rope_table) or None; window, sinks as for bl_attn_decode.  A
    step that finds too few free pages sets `status` (int32 [1], 0 otherwise)
    and leaves the cache and the attention outputs as they were."""

    def __init__(self, layers, gains, M: int, eps: float = 1e-6, record: bool = False, cache=None, seq_ids=None,
                 rope=None, window: int = 0, sinks: int = 0):
        self.M = M
        self.cache = cache
        self.eps = eps
        self.record = record
        self.L = api.lib()
        dev = layers[0]["q"][0].device
        hidden = layers[0]["q"][3]
        ffn = layers[0]["gate"][2]
        self.x0 = torch.zeros(M, hidden, dtype=torch.float32, device=dev)
        self.layers = []
        if cache is not None:
            self._check_cache(layers, hidden, seq_ids, rope)
            self.seq_ids = seq_ids
            self.status = torch.zeros(1, dtype=torch.int32, device=dev)
            self.active = torch.full((M,), -1, dtype=torch.int32, device=dev)
            self._ones = torch.ones(M, dtype=torch.int32, device=dev)
            self._rope = rope
            self._window, self._sinks = window, sinks
            need = api.attn_decode_workspace_bytes(M, hidden // cache.head_dim, cache.kv_heads, cache.head_dim)
            self._workspace = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
        x_in = self.x0
        for li, (lay, (g_o, g_d)) in enumerate(zip(layers, gains)):
            bufs = {}
            for name in PROJ:
                packed, gamma, N, K = lay[name]
                b = dict(packed=packed, gamma=gamma, N=N, K=K,
                         Y=torch.empty(M, N, dtype=torch.float32, device=dev))
                if record:
                    b["x_q"] = torch.empty(M, K, dtype=torch.int8, device=dev)
                    b["s"] = torch.empty(max(M, 4), dtype=torch.float32, device=dev)[:M]
                    b["acc"] = torch.empty(M, N, dtype=torch.int32, device=dev)
                bufs[name] = b
            bufs["ffn_xq"] = torch.empty(M, ffn, dtype=torch.int8, device=dev)
            bufs["ffn_s"] = torch.empty(max(M, 4), dtype=torch.float32, device=dev)[:M]
            bufs["x_in"] = x_in
            bufs["g_o"], bufs["g_d"] = g_o, g_d

            def dec(names, X, gain):
                items = []
                for n in names:
                    b = bufs[n]
                    items.append((b["packed"], b["gamma"], X, gain, b["Y"], b.get("x_q"), b.get("s"), b.get("acc"),
                                  b["N"], b["K"]))
                return api.make_decode_problems(items, M=M), len(items)

            d = bufs["down"]
            bufs["launch_qkv"] = dec(("q", "k", "v"), x_in, None)
            o_in = bufs["q"]["Y"]
            if cache is not None:
                o_in = bufs["attn"] = torch.zeros(M, hidden, dtype=torch.float32, device=dev)
                bufs["q_rot"] = torch.zeros(M, hidden // cache.head_dim, cache.head_dim, dtype=torch.float32, device=dev)
            bufs["launch_o"] = dec(("o",), o_in, g_o)
            bufs["launch_gu"] = dec(("gate", "up"), bufs["o"]["Y"], None)
            bufs["launch_down"] = (api.make_problems([(d["packed"], d["gamma"], bufs["ffn_xq"], bufs["ffn_s"], d["Y"],
                                                       d.get("acc"), d["N"], d["K"])], M=M), 1)
            self.layers.append(bufs)
            x_in = d["Y"]
        self.out = x_in

    def _check_cache(self, layers, hidden: int, seq_ids, rope):
        c = self.cache
        if c.pool.shape[0] != len(layers):
            raise ValueError(f"the cache has {c.pool.shape[0]} layers, the chain {len(layers)}")
        if hidden % c.head_dim or layers[0]["k"][2] != c.kv_heads * c.head_dim:
            raise ValueError(f"projections of {hidden} and {layers[0]['k'][2]} do not make heads of {c.head_dim} "
                             f"over {c.kv_heads} kv heads")
        if not isinstance(seq_ids, torch.Tensor) or seq_ids.dtype != torch.int32 or seq_ids.numel() != self.M:
            raise ValueError(f"seq_ids must be an int32 tensor of {self.M} elements")
        if rope is not None and rope.shape[0] < c.tables.shape[1] * c.page_size:
            raise ValueError(f"rope covers {rope.shape[0]} positions, a sequence may have "
                             f"{c.tables.shape[1] * c.page_size}")

    def launches_per_step(self) -> int:
        """Kernel launches of a step (with a cache: at most; an attention small
        enough for one CTA needs no join)."""
        return 5 * len(self.layers) if self.cache is None else 8 * len(self.layers) + 1

    def _attend(self, li: int, b, stream):
        """q, k, v of layer li -> its attention output (three launches)."""
        c = self.cache
        D = c.head_dim
        kp, vp = c.pages(li)
        q, k, v = (b[n]["Y"].view(self.M, -1, D) for n in ("q", "k", "v"))
        api.bl_rope_append(q, k, v, self._rope, None, c.lengths, self.active, kp, vp, c.tables, q_out=b["q_rot"],
                           stream=stream)
        api.bl_attn_decode(b["q_rot"], kp, vp, c.tables, c.lengths, self.active, self._window, self._sinks,
                           out=b["attn"].view(q.shape), workspace=self._workspace, stream=stream)

    def run(self, stream_ptr: int):
        """Enqueue one token step on the raw stream handle (graph-capturable)."""
        L, M, eps = self.L, self.M, self.eps
        RDY = api.BL_FWD_WEIGHTS_READY
        stream = None
        if self.cache is not None:
            stream = torch.cuda.ExternalStream(stream_ptr) if stream_ptr else torch.cuda.default_stream()
            self.cache.extend(self.seq_ids, self._ones, self.status, self.active, stream)
        for li, b in enumerate(self.layers):
            for key in ("launch_qkv", "launch_o", "launch_gu"):
                arr, n = b[key]
                rc = L.bl_linear_decode_grouped(arr, n, api.BL_F32, M, eps, RDY, stream_ptr)
                if rc:
                    raise api.BitLinearError(rc, "bl_linear_decode_grouped")
                if key == "launch_qkv" and self.cache is not None:
                    self._attend(li, b, stream)
            g, u = b["gate"]["Y"], b["up"]["Y"]
            rc = L.bl_ffn_act_quant(g.data_ptr(), u.data_ptr(), M, g.shape[1], b["g_d"].data_ptr(), eps,
                                    b["ffn_xq"].data_ptr(), b["ffn_s"].data_ptr(), stream_ptr)
            if rc:
                raise api.BitLinearError(rc, "bl_ffn_act_quant")
            arr, n = b["launch_down"]
            rc = L.bl_forward_grouped(arr, n, M, RDY, stream_ptr)
            if rc:
                raise api.BitLinearError(rc, "bl_forward_grouped")
