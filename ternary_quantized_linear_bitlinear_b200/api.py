"""Python binding of libbitlinear.so (include/bitlinear.h, include/bitlinear_attn.h).

Argument marshalling only: every function here checks that torch tensors are
CUDA tensors on the current device, contiguous, of the right dtype and large
enough for the call, allocates outputs with torch when
the caller passes none, and calls the C entry point of the same name with
raw device pointers and the current torch stream.  All arithmetic runs in
the library's kernels; if the library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import struct
import warnings

import torch

from . import build as _build

_LIB = None

BL_F32, BL_BF16 = 0, 1
BL_MAX_GROUP = 128
BL_FWD_WEIGHTS_READY = 1
_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}

_i64 = ctypes.c_int64
_p = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_int = ctypes.c_int


class BitLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class Problem(ctypes.Structure):
    """bl_problem: one (packed, gamma, x_q, s, Y) problem of a grouped forward."""
    _fields_ = [("packed", _p), ("gamma", _p), ("x_q", _p), ("s", _p), ("Y", _p),
                ("acc_out", _p), ("N", _i64), ("K", _i64)]


class ActProblem(ctypes.Structure):
    """bl_act_problem: one activation input of a grouped act quant."""
    _fields_ = [("X", _p), ("subln_gain", _p), ("x_q", _p), ("s", _p), ("K", _i64)]


class WeightProblem(ctypes.Structure):
    """bl_weight_problem: one weight matrix of a grouped weight quantization."""
    _fields_ = [("W", _p), ("N", _i64), ("K", _i64), ("packed", _p), ("gamma", _p)]


class LinearProblem(ctypes.Structure):
    """bl_linear_problem: one weight matrix (and its output) of a grouped bl_linear."""
    _fields_ = [("W", _p), ("Y", _p), ("N", _i64)]


class DecodeProblem(ctypes.Structure):
    """bl_decode_problem: one problem of the fused grouped decode (X in, Y out)."""
    _fields_ = [("packed", _p), ("gamma", _p), ("X", _p), ("subln_gain", _p), ("Y", _p), ("x_q", _p),
                ("s", _p), ("acc_out", _p), ("N", _i64), ("K", _i64)]


class KvCache(ctypes.Structure):
    """bl_kv_cache: the paged cache of one layer, as the kernels see it."""
    _fields_ = [("k_pages", _p), ("v_pages", _p), ("tables", _p), ("lengths", _p), ("num_pages", _i64),
                ("page_size", _i64), ("max_seqs", _i64), ("max_pages", _i64), ("dtype", _int)]


# The same bytes without a Structure object per call (a fifth of its cost).
_KV_CACHE = struct.Struct("PPPPqqqqi4x")
assert _KV_CACHE.size == ctypes.sizeof(KvCache)


_SIGS = {
    "bl_status_string": (ctypes.c_char_p, [_int]),
    "bl_version": (_int, []),
    "bl_check_device_error": (_int, [_p]),
    "bl_quant_weights_workspace_bytes": (_sz, [_i64, _i64]),
    "bl_quant_weights": (_int, [_p, _int, _i64, _i64, _p, _p, _p, _sz, _p]),
    "bl_quant_weights_noalloc": (_int, [_p, _int, _i64, _i64, _p, _p, _p]),
    "bl_quant_act": (_int, [_p, _int, _i64, _i64, _p, _f32, _p, _p, _p]),
    "bl_ffn_act_quant": (_int, [_p, _p, _i64, _i64, _p, _f32, _p, _p, _p]),
    "bl_forward": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p]),
    "bl_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bl_linear": (_int, [_p, _int, _p, _int, _i64, _i64, _i64, _p, _f32, _p, _sz, _p, _p]),
    "bl_forward_grouped": (_int, [ctypes.POINTER(Problem), _int, _i64, ctypes.c_uint, _p]),
    "bl_debug_decode_plan": (_int, [_p, _int, _i64, _int, _p, _int, _p]),
    "bl_debug_forward_prefill": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, ctypes.c_longlong,
                                        ctypes.c_uint32, _p]),
    "bl_quant_act_grouped": (_int, [ctypes.POINTER(ActProblem), _int, _int, _i64, _f32, _p]),
    "bl_linear_decode_grouped": (_int, [ctypes.POINTER(DecodeProblem), _int, _int, _i64, _f32, ctypes.c_uint,
                                        _p]),
    "bl_quant_weights_grouped": (_int, [ctypes.POINTER(WeightProblem), _int, _int, _p, _sz, _p]),
    "bl_forward_glu": (_int, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, _p]),
    "bl_backward_dx": (_int, [_p, _p, _p, _i64, _i64, _i64, _p, _p]),
    "bl_backward_dw_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bl_backward_dw": (_int, [_p, _p, _p, _p, _int, _p, _f32, _i64, _i64, _i64, _p, _sz, _p, _p]),
    "bl_linear_grouped_workspace_bytes": (_sz, [ctypes.POINTER(LinearProblem), _int, _i64, _i64]),
    "bl_linear_grouped": (_int, [ctypes.POINTER(LinearProblem), _int, _int, _p, _int, _i64, _i64, _p, _f32, _p, _sz,
                                 _p]),
    "bl_rope_append": (_int, [_p, _p, _p, _int, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _p, _i64, _int, _p, _i64, _p,
                              _p, _i64, _p, _p, _p, _p, _int, _p]),
    "bl_attn_decode_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "bl_attn_decode": (_int, [_p, _int, _i64, _i64, _i64, _i64, _i64, _p, _p, _i64, _i64, _f32, _p,
                              _sz, _p, _p, _p]),
    "bl_kv_extend": (_int, [_p, _p, _p, _i64, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _p]),
    "bl_kv_free": (_int, [_p, _p, _p, _i64, _i64, _i64, _i64, _p, _i64, _p]),
    "bl_kv_fork_workspace_bytes": (_sz, [_i64]),
    "bl_kv_fork": (_int, [_p, _i64, _i64, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _p, _i64, _p, _sz, _p, _p]),
    "bl_kv_compact_workspace_bytes": (_sz, [_i64]),
    "bl_kv_compact": (_int, [_p, _i64, _i64, _p, _p, _i64, _i64, _i64, _p, _sz, _p, _p]),
    "bl_attn_forward": (_int, [_p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _p, _p, _i64, _i64, _i64,
                               _i64, _i64, _f32, _p, _p, _p]),
    "bl_attn_backward_workspace_bytes": (_sz, [_i64] * 10),
    "bl_attn_backward": (_int, [_p] * 6 + [_i64] * 9 + [_p, _p] + [_i64] * 5 + [_f32, _p, _sz, _p, _p, _p, _p]),
}

EXPORTED = tuple(_SIGS)


# attn_binding.so, once loaded, and what bind() there takes.
_FAST = None
_FAST_ENTRIES = ("bl_rope_append", "bl_attn_decode_workspace_bytes", "bl_attn_decode", "bl_kv_extend", "bl_kv_free",
                 "bl_kv_fork_workspace_bytes", "bl_kv_fork", "bl_kv_compact_workspace_bytes", "bl_kv_compact",
                 "bl_attn_forward", "bl_attn_backward_workspace_bytes", "bl_attn_backward")


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load libbitlinear.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m ternary_quantized_linear_bitlinear_b200.build`")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _load_binding(L)
        _LIB = L
    return _LIB


def _load_binding(L):
    """attn_binding.so, the compiled way to the attention calls, with the
    addresses of L's entry points.  Only a shorter way: where it was not built
    (no host compiler, no torch headers) or was built for another torch, the
    attention calls go through the checks of this file, 5 to 10 us slower, and
    nothing else changes."""
    global _FAST
    path = _build.BINDING
    try:
        spec = importlib.util.spec_from_file_location("attn_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        if module.torch_version != torch.__version__:
            raise ImportError(f"built for torch {module.torch_version}, this is {torch.__version__}")
        module.bind(tuple(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in _FAST_ENTRIES))
        _FAST = module
    except (ImportError, OSError) as e:
        _FAST = None
        warnings.warn(f"{path}: {e}; attention calls take 5 to 10 us longer on the host (build it with "
                      "`python -m ternary_quantized_linear_bitlinear_b200.build`)", RuntimeWarning, stacklevel=3)


def status_string(status: int) -> str:
    return lib().bl_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise BitLinearError(status, where)


def _current_device() -> int:
    return torch.cuda.current_device()


def _stream(stream) -> int:
    """Raw handle of `stream` (default: torch's current stream).  The library
    launches on the current device, so an explicit stream must belong to it."""
    if stream is None:
        # the raw handle of torch.cuda.current_stream(), without building the Stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(_current_device())
    if stream.device_index != _current_device():
        raise ValueError(f"stream belongs to cuda:{stream.device_index}, the current device is "
                         f"cuda:{_current_device()}")
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _is_cuda(t: torch.Tensor) -> bool:
    return t.is_cuda


def _device_index(t: torch.Tensor) -> int:
    return t.device.index


def _dev(t: torch.Tensor, name: str, dtype=None, min_numel: int = 0):
    """A device buffer the library reads or writes: CUDA, on the current
    device (the library launches there, so every buffer of a call lives on
    one GPU), contiguous, of the given dtype and at least min_numel elements
    (so that no kernel touches host memory, another GPU's memory, or runs
    past the end of a caller's buffer)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not _is_cuda(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if _device_index(t) != _current_device():
        raise ValueError(f"{name} lives on cuda:{_device_index(t)}, the current device is cuda:{_current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {min_numel}")
    return t


def _opt(t, name: str, dtype=None, min_numel: int = 0):
    return None if t is None else _dev(t, name, dtype, min_numel)


def _mat(t: torch.Tensor, name: str, cols: int | None = None, rows: int | None = None):
    """A 2-D float32 or bfloat16 input matrix ([N, K] weights or [M, K]
    activations) on the current device, optionally with a fixed column
    (and row) count -> (rows, cols)."""
    _dev(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} has {t.shape[1]} columns, expected {cols}")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {rows}")
    return t.shape[0], t.shape[1]


# -- workspace queries ---------------------------------------------------------

def quant_weights_workspace_bytes(N: int, K: int) -> int:
    return int(lib().bl_quant_weights_workspace_bytes(N, K))


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().bl_linear_workspace_bytes(M, N, K))


# -- step 1 --------------------------------------------------------------------

def bl_quant_weights(W: torch.Tensor, packed=None, gamma=None, workspace=None, stream=None):
    """-> (packed uint8 [N, K/4], gamma float32 [1])."""
    N, K = _mat(W, "W")
    if packed is None:
        packed = torch.empty(N, K // 4, dtype=torch.uint8, device=W.device)
    if gamma is None:
        gamma = torch.empty(4, dtype=torch.float32, device=W.device)[:1]
    if workspace is None:
        workspace = torch.empty(quant_weights_workspace_bytes(N, K), dtype=torch.uint8, device=W.device)
    _dev(packed, "packed", torch.uint8, N * K // 4)
    _dev(gamma, "gamma", torch.float32, 1)
    _dev(workspace, "workspace", torch.uint8)
    rc = lib().bl_quant_weights(W.data_ptr(), _DTYPES.get(W.dtype, -1), N, K, packed.data_ptr(), gamma.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(rc, "bl_quant_weights")
    return packed, gamma


def bl_quant_weights_noalloc(W: torch.Tensor, packed=None, gamma=None, stream=None):
    """bl_quant_weights without a workspace argument: the library's static
    device scratch is used instead (for callers that cannot allocate device
    memory; see include/bitlinear.h).  Outputs are allocated here only when
    the caller passes none."""
    N, K = _mat(W, "W")
    if packed is None:
        packed = torch.empty(N, K // 4, dtype=torch.uint8, device=W.device)
    if gamma is None:
        gamma = torch.empty(4, dtype=torch.float32, device=W.device)[:1]
    _dev(packed, "packed", torch.uint8, N * K // 4)
    _dev(gamma, "gamma", torch.float32, 1)
    rc = lib().bl_quant_weights_noalloc(W.data_ptr(), _DTYPES.get(W.dtype, -1), N, K, packed.data_ptr(),
                                        gamma.data_ptr(), _stream(stream))
    _check(rc, "bl_quant_weights_noalloc")
    return packed, gamma


def bl_quant_weights_grouped(Ws, packed=None, gammas=None, workspace=None, stream=None):
    """Several weight matrices (same dtype) in three launches -> ([packed], [gamma]),
    each as bl_quant_weights(W) would give it."""
    Ws = list(Ws)
    if not 1 <= len(Ws) <= 8:
        raise ValueError("between 1 and 8 weight matrices")
    dtype = Ws[0].dtype
    shapes = [_mat(W, f"Ws[{i}]") for i, W in enumerate(Ws)]
    for i, W in enumerate(Ws):
        _dev(W, f"Ws[{i}]", dtype)
    dev = Ws[0].device
    if packed is None:
        packed = [torch.empty(N, K // 4, dtype=torch.uint8, device=dev) for N, K in shapes]
    if gammas is None:
        gammas = [torch.empty(4, dtype=torch.float32, device=dev)[:1] for _ in Ws]
    if workspace is None:
        workspace = torch.empty(quant_weights_workspace_bytes(1, 64), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8)
    arr = (WeightProblem * len(Ws))()
    for i, ((N, K), W, pk, g) in enumerate(zip(shapes, Ws, packed, gammas)):
        _dev(pk, f"packed[{i}]", torch.uint8, N * K // 4)
        _dev(g, f"gammas[{i}]", torch.float32, 1)
        arr[i] = WeightProblem(W.data_ptr(), N, K, pk.data_ptr(), g.data_ptr())
    rc = lib().bl_quant_weights_grouped(arr, len(Ws), _DTYPES[dtype], workspace.data_ptr(), workspace.numel(),
                                        _stream(stream))
    _check(rc, "bl_quant_weights_grouped")
    return packed, gammas


# -- step 2 --------------------------------------------------------------------

def bl_quant_act(X: torch.Tensor, subln_gain=None, subln_eps: float = 1e-6, x_q=None, s=None, stream=None):
    """-> (x_q int8 [M, K], s float32 [M])."""
    M, K = _mat(X, "X")
    if x_q is None:
        x_q = torch.empty(M, K, dtype=torch.int8, device=X.device)
    if s is None:
        s = torch.empty(M, dtype=torch.float32, device=X.device)
    _dev(x_q, "x_q", torch.int8, M * K)
    _dev(s, "s", torch.float32, M)
    _opt(subln_gain, "subln_gain", torch.float32, K)
    rc = lib().bl_quant_act(X.data_ptr(), _DTYPES.get(X.dtype, -1), M, K, _ptr(subln_gain), subln_eps,
                            x_q.data_ptr(), s.data_ptr(), _stream(stream))
    _check(rc, "bl_quant_act")
    return x_q, s


def bl_quant_act_grouped(items, dtype=torch.bfloat16, subln_eps: float = 1e-6, stream=None):
    """items: list of (X [M, K], gain or None, x_q [M, K], s [M]), same M and dtype."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    arr = (ActProblem * len(items))()
    M = items[0][0].shape[0]
    for i, (X, gain, xq, s) in enumerate(items):
        _mat(X, f"items[{i}].X", rows=M)
        _dev(X, f"items[{i}].X", dtype)
        _opt(gain, f"items[{i}].gain", torch.float32, X.shape[1])
        _dev(xq, f"items[{i}].x_q", torch.int8, M * X.shape[1])
        _dev(s, f"items[{i}].s", torch.float32, M)
        arr[i] = ActProblem(X.data_ptr(), _ptr(gain), xq.data_ptr(), s.data_ptr(), X.shape[1])
    rc = lib().bl_quant_act_grouped(arr, len(items), _DTYPES.get(dtype, -1), M, subln_eps, _stream(stream))
    _check(rc, "bl_quant_act_grouped")


# -- steps 3 + 4 ---------------------------------------------------------------

def bl_ffn_act_quant(gate: torch.Tensor, up: torch.Tensor, subln_gain=None, subln_eps: float = 1e-6, x_q=None, s=None,
                     stream=None):
    """Down-projection input from the gate / up outputs: (x_q int8 [M, F], s [M])
    of relu(gate)^2 * up, after SubLN when a gain is given."""
    _dev(gate, "gate", torch.float32)
    _dev(up, "up", torch.float32)
    if gate.dim() != 2 or gate.shape != up.shape:
        raise ValueError("gate and up must be 2-D [M, F] of the same shape")
    M, F = gate.shape
    if x_q is None:
        x_q = torch.empty(M, F, dtype=torch.int8, device=gate.device)
    if s is None:
        s = torch.empty(max(M, 4), dtype=torch.float32, device=gate.device)[:M]
    _dev(x_q, "x_q", torch.int8, M * F)
    _dev(s, "s", torch.float32, M)
    _opt(subln_gain, "subln_gain", torch.float32, F)
    rc = lib().bl_ffn_act_quant(gate.data_ptr(), up.data_ptr(), M, F, _ptr(subln_gain), subln_eps, x_q.data_ptr(),
                                s.data_ptr(), _stream(stream))
    _check(rc, "bl_ffn_act_quant")
    return x_q, s


def bl_forward(packed, gamma, x_q, s, N: int, Y=None, acc_out=None, stream=None):
    """-> Y float32 [M, N] (acc_out int32 [M, N] filled when given)."""
    M, K = _xq2d(x_q)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=x_q.device)
    _check_forward_args(packed, gamma, s, Y, acc_out, M, N, K)
    rc = lib().bl_forward(packed.data_ptr(), gamma.data_ptr(), x_q.data_ptr(), s.data_ptr(), M, N, K, Y.data_ptr(),
                          _ptr(acc_out), _stream(stream))
    _check(rc, "bl_forward")
    return Y


def _xq2d(x_q):
    _dev(x_q, "x_q", torch.int8)
    if x_q.dim() != 2:
        raise ValueError(f"x_q must be 2-D [M, K], got shape {tuple(x_q.shape)}")
    return x_q.shape[0], x_q.shape[1]


def bl_forward_glu(packed_gate, gamma_gate, packed_up, gamma_up, x_q, s, F: int, h=None, stream=None):
    """h float32 [M, F] = relu(Y_gate)^2 * Y_up of the gate and up projections
    on the shared (x_q, s), from one launch that never stores Y_gate or Y_up."""
    M, K = _xq2d(x_q)
    if h is None:
        h = torch.empty(M, F, dtype=torch.float32, device=x_q.device)
    _dev(packed_gate, "packed_gate", torch.uint8, F * K // 4)
    _dev(packed_up, "packed_up", torch.uint8, F * K // 4)
    _dev(gamma_gate, "gamma_gate", torch.float32, 1)
    _dev(gamma_up, "gamma_up", torch.float32, 1)
    _dev(s, "s", torch.float32, M)
    _dev(h, "h", torch.float32, M * F)
    rc = lib().bl_forward_glu(packed_gate.data_ptr(), gamma_gate.data_ptr(), packed_up.data_ptr(), gamma_up.data_ptr(),
                              x_q.data_ptr(), s.data_ptr(), M, F, K, h.data_ptr(), _stream(stream))
    _check(rc, "bl_forward_glu")
    return h


def bl_backward_dx(dY, packed, gamma, K: int, dX=None, stream=None):
    """dX float32 [M, K] = dY @ (gamma W_q) (straight-through backward of the
    activation), dY bfloat16 [M, N]."""
    _dev(dY, "dY", torch.bfloat16)
    if dY.dim() != 2:
        raise ValueError("dY must be 2-D [M, N]")
    M, N = dY.shape
    if dX is None:
        dX = torch.empty(M, K, dtype=torch.float32, device=dY.device)
    _dev(packed, "packed", torch.uint8, N * K // 4)
    _dev(gamma, "gamma", torch.float32, 1)
    _dev(dX, "dX", torch.float32, M * K)
    rc = lib().bl_backward_dx(dY.data_ptr(), packed.data_ptr(), gamma.data_ptr(), M, N, K, dX.data_ptr(),
                              _stream(stream))
    _check(rc, "bl_backward_dx")
    return dX


def bl_backward_dw(dY, x_q, s, W, gamma, beta: float = 0.0, dW=None, workspace=None, stream=None):
    """dW float32 [N, K] = (dY^T @ (x_q / s)) * scale(W / gamma): the weight
    gradient under the hard (beta <= 0) or soft STE scale; dY bfloat16 [M, N],
    x_q, s from the forward's activation quantization, W the latent weights."""
    _dev(dY, "dY", torch.bfloat16)
    if dY.dim() != 2:
        raise ValueError("dY must be 2-D [M, N]")
    M, N = dY.shape
    Mx, K = _xq2d(x_q)
    if Mx != M:
        raise ValueError("x_q and dY disagree on M")
    _mat(W, "W", cols=K, rows=N)
    _dev(s, "s", torch.float32, M)
    _dev(gamma, "gamma", torch.float32, 1)
    if dW is None:
        dW = torch.empty(N, K, dtype=torch.float32, device=dY.device)
    _dev(dW, "dW", torch.float32, N * K)
    need = int(lib().bl_backward_dw_workspace_bytes(M, N, K))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dY.device)
    _dev(workspace, "workspace", torch.uint8, need)
    rc = lib().bl_backward_dw(dY.data_ptr(), x_q.data_ptr(), s.data_ptr(), W.data_ptr(), _DTYPES[W.dtype],
                              gamma.data_ptr(), float(beta), M, N, K, workspace.data_ptr(), workspace.numel(), dW.data_ptr(),
                              _stream(stream))
    _check(rc, "bl_backward_dw")
    return dW


def _check_forward_args(packed, gamma, s, Y, acc_out, M, N, K):
    _dev(packed, "packed", torch.uint8, N * K // 4)
    _dev(gamma, "gamma", torch.float32, 1)
    _dev(s, "s", torch.float32, M)
    _dev(Y, "Y", torch.float32, M * N)
    _opt(acc_out, "acc_out", torch.int32, M * N)


def _rows_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [M, K] when M is not given")
    return t.shape[0]


def make_problems(items, M: int | None = None):
    """items: list of (packed, gamma, x_q, s, Y, acc_out or None, N, K) -> ctypes
    array for bl_forward_grouped at token count M (default: the first x_q's
    row count).  Every buffer is checked against N, K and M: packed uint8
    >= N*K/4, gamma float32 >= 1, x_q int8 >= M*K, s float32 >= M, Y float32
    and acc_out int32 >= M*N."""
    if M is None:
        M = _rows_of(items[0][2], "items[0].x_q")
    arr = (Problem * len(items))()
    for i, (packed, gamma, xq, s, Y, acc, N, K) in enumerate(items):
        _dev(packed, f"items[{i}].packed", torch.uint8, N * K // 4)
        _dev(gamma, f"items[{i}].gamma", torch.float32, 1)
        _dev(xq, f"items[{i}].x_q", torch.int8, M * K)
        _dev(s, f"items[{i}].s", torch.float32, M)
        _dev(Y, f"items[{i}].Y", torch.float32, M * N)
        _opt(acc, f"items[{i}].acc_out", torch.int32, M * N)
        arr[i] = Problem(packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), s.data_ptr(), Y.data_ptr(),
                         _ptr(acc), N, K)
    arr.bl_M = M
    return arr


def _check_array(problems, count: int, M: int, dtype=None):
    """A problem array built by make_problems / make_decode_problems was
    validated for one M (and dtype): launching it with another, or with more
    problems than it holds, would let a kernel run past a buffer."""
    if count < 0 or count > len(problems):
        raise ValueError(f"count {count} outside the {len(problems)} problems of the array")
    checked_M = getattr(problems, "bl_M", None)
    if checked_M is not None and M != checked_M:
        raise ValueError(f"the problem array was checked for M = {checked_M}, called with M = {M}")
    checked_dt = getattr(problems, "bl_dtype", None)
    if dtype is not None and checked_dt is not None and dtype != checked_dt:
        raise ValueError(f"the problem array was checked for X of {checked_dt}, called with {dtype}")


def bl_forward_grouped(problems, count: int, M: int, flags: int = 0, stream=None):
    """problems: ctypes array from make_problems (built once, launched many times)."""
    _check_array(problems, count, M)
    rc = lib().bl_forward_grouped(problems, count, M, flags, _stream(stream))
    _check(rc, "bl_forward_grouped")


def make_decode_problems(items, M: int | None = None):
    """items: list of (packed, gamma, X, subln_gain or None, Y, x_q or None, s or None, acc_out or None, N, K)
    -> ctypes array for bl_linear_decode_grouped at token count M (default:
    the first X's row count).  Every X must have the first one's dtype
    (float32 or bfloat16); every buffer is checked against N, K and M."""
    if M is None:
        M = _rows_of(items[0][2], "items[0].X")
    dtype = items[0][2].dtype if isinstance(items[0][2], torch.Tensor) else None
    if dtype not in _DTYPES:
        raise ValueError(f"X must be float32 or bfloat16, got {dtype}")
    arr = (DecodeProblem * len(items))()
    for i, (packed, gamma, X, gain, Y, xq, s, acc, N, K) in enumerate(items):
        _dev(packed, f"items[{i}].packed", torch.uint8, N * K // 4)
        _dev(gamma, f"items[{i}].gamma", torch.float32, 1)
        _dev(X, f"items[{i}].X", dtype, M * K)
        _opt(gain, f"items[{i}].subln_gain", torch.float32, K)
        _dev(Y, f"items[{i}].Y", torch.float32, M * N)
        _opt(xq, f"items[{i}].x_q", torch.int8, M * K)
        _opt(s, f"items[{i}].s", torch.float32, M)
        _opt(acc, f"items[{i}].acc_out", torch.int32, M * N)
        arr[i] = DecodeProblem(packed.data_ptr(), gamma.data_ptr(), X.data_ptr(), _ptr(gain), Y.data_ptr(), _ptr(xq),
                               _ptr(s), _ptr(acc), N, K)
    arr.bl_M = M
    arr.bl_dtype = dtype
    return arr


def bl_linear_decode_grouped(problems, count: int, M: int, dtype=torch.bfloat16, subln_eps: float = 1e-6,
                             flags: int = 0, stream=None):
    """Steps 2-4 fused: problems from make_decode_problems (X of `dtype`, same M)."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    _check_array(problems, count, M, dtype)
    rc = lib().bl_linear_decode_grouped(problems, count, _DTYPES[dtype], M, subln_eps, flags, _stream(stream))
    _check(rc, "bl_linear_decode_grouped")


# -- all four steps ------------------------------------------------------------

def bl_linear(W, X, subln_gain=None, subln_eps: float = 1e-6, Y=None, workspace=None, stream=None):
    """-> Y float32 [M, N] = BitLinear(X) with weights W quantized in the call."""
    N, K = _mat(W, "W")
    M, _ = _mat(X, "X", cols=K)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=X.device)
    _dev(Y, "Y", torch.float32, M * N)
    _dev(workspace, "workspace", torch.uint8)
    _opt(subln_gain, "subln_gain", torch.float32, K)
    rc = lib().bl_linear(W.data_ptr(), _DTYPES.get(W.dtype, -1), X.data_ptr(), _DTYPES.get(X.dtype, -1), M, N, K,
                         _ptr(subln_gain), subln_eps, workspace.data_ptr(), workspace.numel(), Y.data_ptr(),
                         _stream(stream))
    _check(rc, "bl_linear")
    return Y


def bl_linear_grouped(Ws, X, subln_gain=None, subln_eps: float = 1e-6, Ys=None, workspace=None, stream=None):
    """Up to 4 weight matrices sharing the input X (e.g. q, k, v), all steps,
    weights quantized in the call -> [Y_i float32 [M, N_i]]."""
    Ws = list(Ws)
    if not 1 <= len(Ws) <= 4:
        raise ValueError("between 1 and 4 weight matrices")
    wdt = Ws[0].dtype
    shapes = [_mat(W, f"Ws[{i}]") for i, W in enumerate(Ws)]
    K = shapes[0][1]
    for i, W in enumerate(Ws):
        _mat(W, f"Ws[{i}]", cols=K)
        _dev(W, f"Ws[{i}]", wdt)
    M, _ = _mat(X, "X", cols=K)
    if Ys is None:
        Ys = [torch.empty(M, N, dtype=torch.float32, device=X.device) for N, _ in shapes]
    arr = (LinearProblem * len(Ws))()
    for i, ((N, _), W, Y) in enumerate(zip(shapes, Ws, Ys)):
        _dev(Y, f"Ys[{i}]", torch.float32, M * N)
        arr[i] = LinearProblem(W.data_ptr(), Y.data_ptr(), N)
    need = int(lib().bl_linear_grouped_workspace_bytes(arr, len(Ws), M, K))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _dev(workspace, "workspace", torch.uint8, need)
    _opt(subln_gain, "subln_gain", torch.float32, K)
    rc = lib().bl_linear_grouped(arr, len(Ws), _DTYPES[wdt], X.data_ptr(), _DTYPES[X.dtype], M, K, _ptr(subln_gain),
                                 subln_eps, workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(rc, "bl_linear_grouped")
    return Ys


# -- attention and its cache (include/bitlinear_attn.h) ------------------------
#
# These calls are a few microseconds of GPU work at decode sizes, so the plain
# valid call is recognised and made by compiled code (_FAST,
# csrc/attn_binding.cpp).  What it does not take comes back as None and goes
# through the checks here.

_Tensor = torch.Tensor
_I32 = torch.int32


def _ok(t, dtype, cur: int) -> bool:
    # (get_device() is -1 for a CPU tensor)
    return isinstance(t, _Tensor) and t.get_device() == cur and t.dtype is dtype and t.is_contiguous()


def _rows3(t, name: str, cur: int, heads: int | None = None, D: int | None = None, dtype=None, rows: int | None = None):
    """Rows of heads [T, H, D] on the current device whose heads are contiguous
    (a row may be part of a wider one) -> row stride in elements."""
    if isinstance(t, _Tensor) and t.get_device() == cur and len(t.shape) == 3:
        T, H, d = t.shape
        st, sh, sd = t.stride()
        dt = t.dtype
        if (sd == 1 and (sh == d or H == 1) and (dt is dtype or (dtype is None and dt in _DTYPES))
                and (rows is None or T == rows) and (heads is None or H == heads) and (D is None or d == D)):
            if T == 1:
                return H * d
            if st >= H * d:
                return st
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [T, heads, D], got shape {tuple(t.shape)}")
    if not _is_cuda(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if _device_index(t) != _current_device():
        raise ValueError(f"{name} lives on cuda:{_device_index(t)}, the current device is cuda:{_current_device()}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    T, H, d = t.shape
    for what, got, want in (("rows", T, rows), ("heads", H, heads), ("as head size", d, D)):
        if want is not None and got != want:
            raise ValueError(f"{name} has {got} {what}, expected {want}")
    if (d > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride = t.stride(0) if T > 1 else H * d
    if stride < H * d:
        raise ValueError(f"{name}: rows overlap (stride {stride}, {H * d} elements each)")
    return stride


def _on(stream, fn, *args):
    """fn(*args) with `stream` current: what the call allocates then belongs to
    the stream it is used on (memory of another stream's pool may still be in
    use there, or be handed out again before this call's kernels have run)."""
    _stream(stream)  # of the current device?
    with torch.cuda.stream(stream):
        return fn(*args)


def _answer(done, where: str):
    """What _FAST returned: the results, or the status of a call that was refused."""
    if done.__class__ is int:
        _check(done, where)
    return done


def _buf(t, name: str, dtype, min_numel: int, cur: int):
    if not (_ok(t, dtype, cur) and t.numel() >= min_numel):
        _dev(t, name, dtype, min_numel)
    return t.data_ptr()


def _i32(t, name: str, numel: int, cur: int):
    """An int32 buffer of exactly numel elements -> its address."""
    if not (_ok(t, torch.int32, cur) and t.numel() == numel):
        _dev(t, name, torch.int32)
        if t.numel() != numel:
            raise ValueError(f"{name} holds {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _tables2(tables, lengths, refs, cur: int):
    """Checked tables [max_seqs, max_pages], lengths [max_seqs] and refs
    [num_pages] (either may be None) -> (max_seqs, max_pages)."""
    if not (_ok(tables, _I32, cur) and len(tables.shape) == 2):
        _dev(tables, "tables", torch.int32)
        if tables.dim() != 2:
            raise ValueError("tables must be 2-D [max_seqs, max_pages]")
    max_seqs, max_pages = tables.shape
    if lengths is not None and not (_ok(lengths, _I32, cur) and lengths.numel() == max_seqs):
        _i32(lengths, "lengths", max_seqs, cur)
    if refs is not None and not (_ok(refs, _I32, cur) and len(refs.shape) == 1):
        _dev(refs, "refs", torch.int32)
        if refs.dim() != 1:
            raise ValueError("refs must be 1-D [num_pages]")
    return max_seqs, max_pages


def _kv_cache(k_pages, v_pages, tables, lengths, heads, D: int, cur: int):
    """The bytes of a bl_kv_cache of checked pages [num_pages, Hkv, page_size, D]
    and tables -> (bytes, Hkv, max_seqs)."""
    dt = k_pages.dtype if isinstance(k_pages, _Tensor) else None
    shape = k_pages.shape if dt in _DTYPES else ()
    if not (len(shape) == 4 and isinstance(v_pages, _Tensor) and k_pages.get_device() == cur
            and v_pages.get_device() == cur and v_pages.dtype is dt and v_pages.shape == shape
            and k_pages.is_contiguous() and v_pages.is_contiguous()):
        _dev(k_pages, "k_pages")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be 4-D [num_pages, Hkv, page_size, D]")
        if dt not in _DTYPES:
            raise ValueError(f"k_pages must be float32 or bfloat16, got {dt}")
        _dev(v_pages, "v_pages", dt)
        if v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages must have the same shape")
        shape = k_pages.shape
    pages, Hkv, ps, d = shape
    if heads is not None and Hkv != heads:
        raise ValueError(f"the pages have {Hkv} heads, expected {heads}")
    if d != D:
        raise ValueError(f"the pages have head size {d}, expected {D}")
    max_seqs, max_pages = _tables2(tables, lengths, None, cur)
    return _KV_CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), tables.data_ptr(), lengths.data_ptr(), pages, ps,
                          max_seqs, max_pages, _DTYPES[dt]), Hkv, max_seqs


def bl_rope_append(q=None, k=None, v=None, rope=None, cu_seqlens=None, lengths=None, seq_ids=None, k_pages=None,
                   v_pages=None, tables=None, out_dtype=None, q_out=None, k_out=None, v_out=None, keep_kv=None,
                   inverse: bool = False, stream=None):
    """Rotary positions on q [T, Hq, D] and k [T, Hkv, D], rounded to out_dtype
    (default: q's dtype), and k, v into their pages when pages are given ->
    (q_out, k_out, v_out).  k_out and v_out are made when no pages are given
    or keep_kv is set.  rope [positions, D] float32: cos of D/2 angles, then
    sin.  Batch entry b's tokens are rows cu_seqlens[b] .. cu_seqlens[b+1] - 1
    (one row each without cu_seqlens) and stand at the end of sequence
    seq_ids[b] (default b) of lengths[seq] tokens; without lengths they stand
    at 0, 1, ...  inverse=True rotates back (the gradient).  An output may be
    the very tensor it comes from (same dtype, same rows), not overlap it
    otherwise."""
    if stream is not None:
        return _on(stream, bl_rope_append, q, k, v, rope, cu_seqlens, lengths, seq_ids, k_pages, v_pages, tables, out_dtype,
                   q_out, k_out, v_out, keep_kv, inverse)
    if _FAST is not None:
        done = _FAST.rope_append(q, k, v, rope, cu_seqlens, lengths, seq_ids, k_pages, v_pages, tables, out_dtype, q_out,
                                 k_out, v_out, keep_kv, inverse)
        if done is not None:
            return _answer(done, "bl_rope_append")
    cur = _current_device()
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    if not isinstance(first, _Tensor) or first.dim() != 3:
        raise ValueError("q, k and v must be 3-D tensors [T, heads, D]")
    T, Hq, D = first.shape
    dt = first.dtype
    qs = ks = vs = 0
    if q is not None:
        qs = _rows3(q, "q", cur, dtype=dt)
    Hkv = Hq
    if (k is None) != (v is None):
        raise ValueError("k and v must be given together")
    if k is not None:
        ks = _rows3(k, "k", cur, D=D, dtype=dt, rows=T)
        Hkv = k.shape[1]
        vs = _rows3(v, "v", cur, heads=Hkv, D=D, dtype=dt, rows=T)
    odt = dt if out_dtype is None else out_dtype
    if odt not in _DTYPES:
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {odt}")
    B = T
    if cu_seqlens is not None:
        _buf(cu_seqlens, "cu_seqlens", torch.int32, 2, cur)
        B = cu_seqlens.numel() - 1
    if seq_ids is not None:
        _i32(seq_ids, "seq_ids", B, cur)
    if rope is not None and not (_ok(rope, torch.float32, cur) and rope.dim() == 2 and rope.shape[1] == D):
        _dev(rope, "rope", torch.float32)
        if rope.dim() != 2 or rope.shape[1] != D:
            raise ValueError(f"rope must be [positions, {D}]")
    cache = None
    max_seqs = 0
    if (k_pages is None) != (v_pages is None):
        raise ValueError("k_pages and v_pages must be given together")
    if k_pages is not None:
        if k is None or tables is None or lengths is None:
            raise ValueError("pages need k, v, tables and lengths")
        cache, _, max_seqs = _kv_cache(k_pages, v_pages, tables, lengths, Hkv, D, cur)
    elif lengths is not None:
        _buf(lengths, "lengths", torch.int32, 1, cur)
        max_seqs = lengths.numel()
    if lengths is not None and seq_ids is None and B > max_seqs:
        raise ValueError(f"{B} batch entries, but lengths holds {max_seqs} sequences")
    if q is not None:
        if q_out is None:
            q_out = q.new_empty((T, Hq, D)) if odt is dt else q.new_empty((T, Hq, D), dtype=odt)
        else:
            _buf(q_out, "q_out", odt, T * Hq * D, cur)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is None:
        if k_out is not None or v_out is not None:
            raise ValueError("k_out or v_out without k and v")
    else:
        if (cache is None) if keep_kv is None else keep_kv:
            k_out = k.new_empty((T, Hkv, D), dtype=odt) if k_out is None else k_out
            v_out = k.new_empty((T, Hkv, D), dtype=odt) if v_out is None else v_out
        if k_out is not None:
            _buf(k_out, "k_out", odt, T * Hkv * D, cur)
        if v_out is not None:
            _buf(v_out, "v_out", odt, T * Hkv * D, cur)
    rc = lib().bl_rope_append(_ptr(q), _ptr(k), _ptr(v), _DTYPES[dt], qs, ks, vs, T, Hq, Hkv, D, _ptr(rope),
                              0 if rope is None else rope.shape[0], int(inverse), _ptr(cu_seqlens), B, _ptr(seq_ids),
                              None if cache is not None else _ptr(lengths), max_seqs, cache, _ptr(q_out), _ptr(k_out),
                              _ptr(v_out), _DTYPES[odt], _stream(None))
    if rc:
        _check(rc, "bl_rope_append")
    return q_out, k_out, v_out


def attn_decode_workspace_bytes(B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().bl_attn_decode_workspace_bytes(B, Hq, Hkv, D))


def bl_attn_decode(q, k_pages, v_pages, tables, lengths, seq_ids=None, window: int = 0, sinks: int = 0, scale=None,
                   out=None, lse=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of one new token per sequence over the paged cache -> out
    [B, Hq, D] of q's dtype (and lse float32 [B, Hq] with return_lse=True).
    Entry b reads sequence seq_ids[b] (default b); window = 0 sees all keys,
    otherwise the last `window` and the first `sinks`; scale defaults to
    D ** -0.5.  Calls that may run at the same time need workspaces of their
    own (the default: a new one per call)."""
    if stream is not None:
        return _on(stream, bl_attn_decode, q, k_pages, v_pages, tables, lengths, seq_ids, window, sinks, scale, out, lse,
                   return_lse, workspace)
    if _FAST is not None:
        done = _FAST.attn_decode(q, k_pages, v_pages, tables, lengths, seq_ids, window, sinks, scale, out, lse,
                                 return_lse, workspace)
        if done is not None:
            return _answer(done, "bl_attn_decode")
    cur = _current_device()
    qs = _rows3(q, "q", cur)
    B, Hq, D = q.shape
    cache, Hkv, max_seqs = _kv_cache(k_pages, v_pages, tables, lengths, None, D, cur)
    if seq_ids is not None:
        _i32(seq_ids, "seq_ids", B, cur)
    elif B > max_seqs:
        raise ValueError(f"{B} batch entries, but the tables hold {max_seqs} sequences")
    if out is None:
        out = q.new_empty((B, Hq, D))
    else:
        _buf(out, "out", q.dtype, B * Hq * D, cur)
    if lse is not None:
        _buf(lse, "lse", torch.float32, B * Hq, cur)
    elif return_lse:
        lse = q.new_empty((B, Hq), dtype=torch.float32)
    L = lib()
    if workspace is None:
        workspace = tables.new_empty(L.bl_attn_decode_workspace_bytes(B, Hq, Hkv, D) // 4 or 16)
    else:
        _buf(workspace, "workspace", torch.uint8, 1, cur)
    rc = L.bl_attn_decode(q.data_ptr(), _DTYPES[q.dtype], qs, B, Hq, Hkv, D, cache, _ptr(seq_ids), window, sinks,
                          D ** -0.5 if scale is None else scale, workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), out.data_ptr(), _ptr(lse), _stream(None))
    if rc:
        _check(rc, "bl_attn_decode")
    return (out, lse) if return_lse else out


def _status(status, like, cur: int):
    if status is None:
        return like.new_empty(1)
    _buf(status, "status", torch.int32, 1, cur)
    return status


def bl_kv_extend(tables, lengths, refs, seq_ids, counts, page_size: int, status=None, active=None, stream=None):
    """Sequence seq_ids[i] grows by counts[i] tokens: pages from the lowest free
    ones, lengths raised -> status int32 [1] (0: done; otherwise nothing was
    changed, see bitlinear_attn.h).  active int32 [n], when given, becomes
    seq_ids, or -1 throughout when the call failed."""
    if stream is not None:
        return _on(stream, bl_kv_extend, tables, lengths, refs, seq_ids, counts, page_size, status, active)
    if _FAST is not None:
        done = _FAST.kv_extend(tables, lengths, refs, seq_ids, counts, page_size, status, active)
        if done is not None:
            return _answer(done, "bl_kv_extend")
    cur = _current_device()
    max_seqs, max_pages = _tables2(tables, lengths, refs, cur)
    ids = _buf(seq_ids, "seq_ids", torch.int32, 1, cur)
    n = seq_ids.numel()
    cnt = _i32(counts, "counts", n, cur)
    status = _status(status, tables, cur)
    if active is not None:
        _i32(active, "active", n, cur)
    rc = lib().bl_kv_extend(tables.data_ptr(), lengths.data_ptr(), refs.data_ptr(), refs.numel(), page_size, max_seqs,
                            max_pages, ids, cnt, n, status.data_ptr(), _ptr(active), _stream(None))
    if rc:
        _check(rc, "bl_kv_extend")
    return status


def bl_kv_free(tables, lengths, refs, seq_ids, page_size: int, stream=None):
    """The sequences end: their pages' refs fall by one, rows become -1, lengths 0."""
    if stream is not None:
        return _on(stream, bl_kv_free, tables, lengths, refs, seq_ids, page_size)
    if _FAST is not None:
        done = _FAST.kv_free(tables, lengths, refs, seq_ids, page_size)
        if done is not None:
            return None if done == 0 else _answer(done, "bl_kv_free")
    cur = _current_device()
    max_seqs, max_pages = _tables2(tables, lengths, refs, cur)
    ids = _buf(seq_ids, "seq_ids", torch.int32, 1, cur)
    rc = lib().bl_kv_free(tables.data_ptr(), lengths.data_ptr(), refs.data_ptr(), refs.numel(), page_size, max_seqs,
                          max_pages, ids, seq_ids.numel(), _stream(None))
    if rc:
        _check(rc, "bl_kv_free")


def _pool(pool, refs, cur: int):
    """A pool [..., num_pages, Hkv, page_size, D] -> (planes, bytes of a page, page size)."""
    dt = pool.dtype if isinstance(pool, _Tensor) else None
    if not (dt in _DTYPES and _ok(pool, dt, cur)):
        _dev(pool, "pool")
        if dt not in _DTYPES:
            raise ValueError(f"pool must be float32 or bfloat16, got {dt}")
    shape = pool.shape
    if len(shape) < 4 or shape[-4] != refs.numel():
        raise ValueError("pool must be [..., num_pages, Hkv, page_size, D] with refs' number of pages")
    return math.prod(shape[:-4]), shape[-3] * shape[-2] * shape[-1] * pool.element_size(), shape[-2]


def bl_kv_fork(pool, tables, lengths, refs, src, dst, status=None, workspace=None, stream=None):
    """Sequence dst[i] (empty) becomes a copy of src[i]: full pages are shared, a
    last partial page is copied in every plane of pool [..., num_pages, Hkv,
    page_size, D] -> status int32 [1], as for bl_kv_extend."""
    if stream is not None:
        return _on(stream, bl_kv_fork, pool, tables, lengths, refs, src, dst, status, workspace)
    if _FAST is not None:
        done = _FAST.kv_fork(pool, tables, lengths, refs, src, dst, status, workspace)
        if done is not None:
            return _answer(done, "bl_kv_fork")
    cur = _current_device()
    max_seqs, max_pages = _tables2(tables, lengths, refs, cur)
    planes, page_bytes, ps = _pool(pool, refs, cur)
    a = _buf(src, "src", torch.int32, 1, cur)
    n = src.numel()
    b = _i32(dst, "dst", n, cur)
    status = _status(status, tables, cur)
    L = lib()
    if workspace is None:
        workspace = tables.new_empty(L.bl_kv_fork_workspace_bytes(n) // 4 or 4)
    else:
        _buf(workspace, "workspace", torch.uint8, 1, cur)
    rc = L.bl_kv_fork(pool.data_ptr(), planes, page_bytes, tables.data_ptr(), lengths.data_ptr(), refs.data_ptr(),
                      refs.numel(), ps, max_seqs, max_pages, a, b, n, workspace.data_ptr(),
                      workspace.numel() * workspace.element_size(), status.data_ptr(), _stream(None))
    if rc:
        _check(rc, "bl_kv_fork")
    return status


def bl_kv_compact(pool, tables, refs, n_live=None, workspace=None, stream=None):
    """The pages in use move to the lowest numbers, in every plane of pool;
    tables and refs follow -> n_live int32 [1], the pages in use."""
    if stream is not None:
        return _on(stream, bl_kv_compact, pool, tables, refs, n_live, workspace)
    if _FAST is not None:
        done = _FAST.kv_compact(pool, tables, refs, n_live, workspace)
        if done is not None:
            return _answer(done, "bl_kv_compact")
    cur = _current_device()
    max_seqs, max_pages = _tables2(tables, None, refs, cur)
    planes, page_bytes, _ = _pool(pool, refs, cur)
    if n_live is None:
        n_live = tables.new_empty(1)
    else:
        _buf(n_live, "n_live", torch.int32, 1, cur)
    L = lib()
    pages = refs.numel()
    if workspace is None:
        workspace = tables.new_empty(L.bl_kv_compact_workspace_bytes(pages) // 4 or 4)
    else:
        _buf(workspace, "workspace", torch.uint8, 1, cur)
    rc = L.bl_kv_compact(pool.data_ptr(), planes, page_bytes, tables.data_ptr(), refs.data_ptr(), pages, max_seqs,
                         max_pages, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         n_live.data_ptr(), _stream(None))
    if rc:
        _check(rc, "bl_kv_compact")
    return n_live


def _ragged(q, k, v, cu_q, cu_k, cur: int):
    b16 = torch.bfloat16
    qs = _rows3(q, "q", cur, dtype=b16)
    Tq, Hq, D = q.shape
    ks = _rows3(k, "k", cur, D=D, dtype=b16)
    Tk, Hkv, _ = k.shape
    vs = _rows3(v, "v", cur, heads=Hkv, D=D, dtype=b16, rows=Tk)
    a = _buf(cu_q, "cu_q", torch.int32, 2, cur)
    n = cu_q.numel()
    return (qs, ks, vs), (Tq, Tk, Hq, Hkv, D), (a, _i32(cu_k, "cu_k", n, cur), n - 1)


def bl_attn_forward(q, k, v, cu_q, cu_k, max_q: int, max_k: int, window: int = 0, sinks: int = 0, scale=None, o=None,
                    lse=None, stream=None):
    """Causal attention over a ragged batch, bfloat16: q [Tq, Hq, D], k, v
    [Tk, Hkv, D]; entry b's queries are rows cu_q[b] .. cu_q[b+1] - 1 and its
    keys cu_k[b] .. cu_k[b+1] - 1, the last query standing at the last key.
    window = 0 sees every earlier key, otherwise the last `window` and the
    first `sinks` -> (o bfloat16 [Tq, Hq, D], lse float32 [Hq, Tq])."""
    if stream is not None:
        return _on(stream, bl_attn_forward, q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale, o, lse)
    if _FAST is not None:
        done = _FAST.attn_forward(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale, o, lse)
        if done is not None:
            return _answer(done, "bl_attn_forward")
    cur = _current_device()
    strides, (Tq, Tk, Hq, Hkv, D), (a, b, B) = _ragged(q, k, v, cu_q, cu_k, cur)
    if o is None:
        o = q.new_empty((Tq, Hq, D))
    else:
        _buf(o, "o", torch.bfloat16, Tq * Hq * D, cur)
    if lse is None:
        lse = q.new_empty((Hq, Tq), dtype=torch.float32)
    else:
        _buf(lse, "lse", torch.float32, Hq * Tq, cur)
    rc = lib().bl_attn_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, Tq, Tk, Hq, Hkv, D, a, b, B, max_q,
                               max_k, window, sinks, D ** -0.5 if scale is None else scale, o.data_ptr(),
                               lse.data_ptr(), _stream(None))
    if rc:
        _check(rc, "bl_attn_forward")
    return o, lse


def bl_attn_backward(do, q, k, v, o, lse, cu_q, cu_k, max_q: int, max_k: int, window: int = 0, sinks: int = 0,
                     scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of bl_attn_forward (o, lse its outputs; do bfloat16 [Tq, Hq, D])
    -> (dq [Tq, Hq, D], dk, dv [Tk, Hkv, D]) bfloat16; dk and dv sum over the
    query heads that share a head."""
    if stream is not None:
        return _on(stream, bl_attn_backward, do, q, k, v, o, lse, cu_q, cu_k, max_q, max_k, window, sinks, scale, dq, dk, dv,
                   workspace)
    if _FAST is not None:
        done = _FAST.attn_backward(do, q, k, v, o, lse, cu_q, cu_k, max_q, max_k, window, sinks, scale, dq, dk, dv,
                                   workspace)
        if done is not None:
            return _answer(done, "bl_attn_backward")
    cur = _current_device()
    b16 = torch.bfloat16
    strides, (Tq, Tk, Hq, Hkv, D), (a, b, B) = _ragged(q, k, v, cu_q, cu_k, cur)
    dos = _rows3(do, "do", cur, heads=Hq, D=D, dtype=b16, rows=Tq)
    _buf(o, "o", b16, Tq * Hq * D, cur)
    _buf(lse, "lse", torch.float32, Hq * Tq, cur)
    if dq is None:
        dq = q.new_empty((Tq, Hq, D))
    else:
        _buf(dq, "dq", b16, Tq * Hq * D, cur)
    if dk is None:
        dk = k.new_empty((Tk, Hkv, D))
    else:
        _buf(dk, "dk", b16, Tk * Hkv * D, cur)
    if dv is None:
        dv = v.new_empty((Tk, Hkv, D))
    else:
        _buf(dv, "dv", b16, Tk * Hkv * D, cur)
    L = lib()
    if workspace is None:
        need = L.bl_attn_backward_workspace_bytes(Tq, Tk, Hq, Hkv, D, B, max_q, max_k, window, sinks)
        workspace = cu_q.new_empty(need // 4 or 4)
    else:
        _buf(workspace, "workspace", torch.uint8, 1, cur)
    rc = L.bl_attn_backward(do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dos,
                            *strides, Tq, Tk, Hq, Hkv, D, a, b, B, max_q, max_k, window, sinks,
                            D ** -0.5 if scale is None else scale, workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _stream(None))
    if rc:
        _check(rc, "bl_attn_backward")
    return dq, dk, dv


def bl_debug_decode_plan(shapes, M: int, sms: int = 148):
    """Host-side plan of a decode call over problems of the given (N, K)
    shapes at M tokens on a GPU with `sms` SMs (nothing is launched; no GPU
    needed): a list of launches, each {"ctas", "smem", "problems": [{"job",
    "row0", "rows", "glog", "kch", "cta_begin"}]}."""
    shapes = list(shapes)
    arr = (ctypes.c_int64 * (2 * len(shapes)))(*[int(v) for nk in shapes for v in nk])
    cap = 64 + 16 * 6 * max(1, len(shapes)) * 8
    out = (ctypes.c_int * cap)()
    written = ctypes.c_int(0)
    rc = lib().bl_debug_decode_plan(arr, len(shapes), int(M), int(sms), out, cap, ctypes.byref(written))
    _check(rc, "bl_debug_decode_plan")
    vals, launches, i = list(out[:written.value]), [], 0
    while i < len(vals):
        ctas, smem, n = vals[i:i + 3]
        i += 3
        probs = []
        for _ in range(n):
            job, row0, rows, glog, kch, cta0 = vals[i:i + 6]
            i += 6
            probs.append(dict(job=job, row0=row0, rows=rows, glog=glog, kch=kch, cta_begin=cta0))
        launches.append(dict(ctas=ctas, smem=smem, problems=probs))
    return launches


def bl_debug_forward_prefill(packed, gamma, x_q, s, N: int, Y=None, acc_out=None, skip_iter: int = -1,
                             timeout_us: int = 2_000_000, stream=None):
    """Test hook (include/bitlinear_debug.h): bl_forward forced through the
    tcgen05 prefill engine, with bounded waits of timeout_us and an optional
    stalled k-iteration."""
    M, K = _xq2d(x_q)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=x_q.device)
    _check_forward_args(packed, gamma, s, Y, acc_out, M, N, K)
    rc = lib().bl_debug_forward_prefill(packed.data_ptr(), gamma.data_ptr(), x_q.data_ptr(), s.data_ptr(), M, N, K,
                                        Y.data_ptr(), _ptr(acc_out), skip_iter, timeout_us, _stream(stream))
    _check(rc, "bl_debug_forward_prefill")
    return Y


def bl_check_device_error(stream=None):
    _check(lib().bl_check_device_error(_stream(stream)), "bl_check_device_error")
