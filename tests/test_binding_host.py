"""Which file each entry point needs, and what building makes (no GPU)."""
import os

import pytest
import torch

from mixture_experts_layer_07_gb300 import build as build_mod


@pytest.fixture
def ops(monkeypatch):
    """The module as it is before its first call."""
    build_mod.build()
    from mixture_experts_layer_07_gb300 import ops as o
    monkeypatch.setattr(o, "_L", None)
    monkeypatch.setattr(o, "_B", None)
    return o


def test_the_ctypes_entry_points_need_the_library_alone(ops, monkeypatch, tmp_path):
    missing = str(tmp_path / "no_module.so")
    monkeypatch.setattr(ops, "BINDING_PATH", missing)
    assert ops.workspace_bytes(ops.make_config(64, 256, 8, 2, 128)) > 0
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match=missing):
        ops.add_rmsnorm(x, x[0], 1e-6, x)


def test_a_missing_library_is_named(ops, monkeypatch, tmp_path):
    missing = str(tmp_path / "no_library.so")
    monkeypatch.setattr(ops, "LIB_PATH", missing)
    with pytest.raises(RuntimeError, match=missing):
        ops.workspace_bytes(ops.make_config(64, 256, 8, 2, 128))


def test_without_python_headers_the_library_is_built(monkeypatch, tmp_path, capsys):
    build_mod.build()
    target = str(tmp_path / "module.so")
    monkeypatch.setattr(build_mod, "BINDING", target)
    monkeypatch.setattr(build_mod.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert os.path.exists(build_mod.build())
    assert not os.path.exists(target) and target in capsys.readouterr().err


def test_the_operators_still_reach_the_library(ops):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: a tensor on the GPU"):
        ops.add_rmsnorm(x, x[0].clone(), 1e-6, torch.zeros_like(x))
    with pytest.raises(ops.MoEError):
        ops.add_rmsnorm_backward_scratch_bytes(4, 20)


def test_the_module_of_another_interpreter_is_not_taken_for_this_one(ops):
    """The file's name carries the ABI that it was compiled for."""
    import sysconfig
    assert ops.BINDING_PATH == build_mod.BINDING
    assert build_mod.BINDING.endswith("_moe_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.basename(build_mod.BINDING) != "_moe_binding.so"
