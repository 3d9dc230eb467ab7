"""The compiled binding is an extra: the library builds without it, and calls find their way without it (no GPU needed)."""
import sys

import pytest
import torch

from tile_sparse_gemm_b200 import build as tsg_build
from tile_sparse_gemm_b200 import decoder as dec
import tile_sparse_gemm_b200 as tsg


def test_the_library_is_built_where_the_extension_cannot_be(monkeypatch, tmp_path, capsys):
    built = []
    monkeypatch.setattr(tsg_build, "LIB", tmp_path / "libpatch.so")
    monkeypatch.setattr(tsg_build, "BINDING", tmp_path / "_decoder_binding.so")
    monkeypatch.setattr(tsg_build.subprocess, "run", lambda cmd, **k: built.append(cmd) or (tmp_path / cmd[cmd.index("-o") + 1]).touch())
    monkeypatch.setattr(tsg_build, "PKG", tmp_path)
    monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))  # no CUDA, no headers
    assert tsg_build.build() == tmp_path / "libpatch.so" and (tmp_path / "libpatch.so").exists()
    assert built and all("nvcc" in cmd[0] for cmd in built)
    assert "libtorch_cuda.so" in capsys.readouterr().err


def test_calls_without_the_extension(monkeypatch):
    tsg_build.build()
    monkeypatch.setattr(dec, "_binding", None)
    monkeypatch.delattr(tsg, "_decoder_binding", raising=False)
    monkeypatch.setitem(sys.modules, "tile_sparse_gemm_b200._decoder_binding", None)
    taken = []
    monkeypatch.setattr(dec, "_cuda", lambda t, name: t.device)
    monkeypatch.setattr(dec, "_call", lambda name, *a, **k: taken.append(name))
    q, pos = torch.ones(3, 4, 64, dtype=torch.bfloat16), torch.ones(3, dtype=torch.int32)
    with pytest.warns(UserWarning, match="compiled binding"):
        tsg.patch_rope(q, None, pos, torch.ones(8, 32, 2))
    w = tsg.Weight4(torch.ones(6, 32, dtype=torch.uint8), torch.ones(6, 1, dtype=torch.bfloat16), 64)
    assert tsg.patch_gemm4(torch.ones(2, 64, dtype=torch.bfloat16), w).shape == (2, 6)
    assert taken == ["patch_rope", "patch_gemm4"]
