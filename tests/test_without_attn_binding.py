"""The library without attn_binding.so, which only shortens the attention calls' way from torch."""
from __future__ import annotations

import os

import pytest
import torch

from ternary_quantized_linear_bitlinear_b200 import api, build


@pytest.fixture
def unloaded(monkeypatch):
    """api as before its first call (what was loaded comes back afterwards)."""
    build.build()
    api.lib()
    monkeypatch.setattr(api, "_LIB", None)
    monkeypatch.setattr(api, "_FAST", None)


def refuses_as_ever():
    """Both kinds of call reach their checks."""
    assert api.status_string(0) == "BL_OK"
    assert api._FAST is None
    assert api.attn_decode_workspace_bytes(4, 12, 4, 64) > 0
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        api.bl_rope_append(torch.zeros(4, 6, 64))


@pytest.mark.parametrize("content", [None, b"", b"not a library"])
def test_missing_or_broken(unloaded, monkeypatch, tmp_path, content):
    path = tmp_path / "attn_binding.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(build, "BINDING", str(path))
    with pytest.warns(RuntimeWarning, match="attn_binding"):
        api.lib()
    refuses_as_ever()


def test_of_another_torch(unloaded, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.warns(RuntimeWarning, match="built for torch"):
        api.lib()
    monkeypatch.undo()


def test_present(unloaded):
    api.lib()
    assert api._FAST.torch_version == torch.__version__


@pytest.mark.parametrize("compiler", ["/nonexistent/c++", "false"])
def test_build_without_a_host_compiler(monkeypatch, tmp_path, compiler):
    """The library is built and stays; an older binding does not."""
    build.build()
    path = tmp_path / "attn_binding.so"
    path.write_bytes(b"old")
    os.utime(path, (1, 1))
    monkeypatch.setattr(build, "BINDING", str(path))
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(RuntimeWarning, match="attn_binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not path.exists()


@pytest.mark.gpu
def test_attention_call(unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "attn_binding.so"))
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(9, 2, 64, generator=g).bfloat16().cuda() for _ in range(3))
    cu = torch.tensor([0, 9], dtype=torch.int32).cuda()
    with pytest.warns(RuntimeWarning, match="attn_binding"):
        o, _ = api.bl_attn_forward(q, k, v, cu, cu, 9, 9)
    api.bl_check_device_error()
    s = torch.einsum("ihd,jhd->hij", q.double(), k.double()) / 8
    s = s.masked_fill(torch.ones(9, 9, device="cuda").triu(1).bool(), -torch.inf)
    ref = torch.einsum("hij,jhd->ihd", s.softmax(-1), v.double())
    assert bool(((o - ref).abs() <= 2.0 ** -6 * v.double().abs().max()).all())
