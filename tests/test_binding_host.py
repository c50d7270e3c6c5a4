"""The native module belongs to one torch: another one gets an error, not a call through another C++
interface, and a build makes the module anew (no GPU needed)."""
import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from bf16_activations_nvfp4_b200 import build


def test_module_of_another_torch_is_refused(monkeypatch):
    assert fi._load_binding().torch_version == torch.__version__
    monkeypatch.setattr(fi, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="another torch"):
        fi.quantize_fp8(torch.zeros((4, 64)))
    assert fi._native is None


def test_another_torch_needs_another_module(monkeypatch, tmp_path):
    record = " ".join(build._binding_command(build._nvcc(), build.BINDING))
    monkeypatch.setattr(build, "_stale", lambda target, sources: False)  # by its age alone it would do
    monkeypatch.setattr(build, "BINDING_RECORD", str(tmp_path / "command"))
    assert build._binding_stale(record)
    (tmp_path / "command").write_text(record)
    assert not build._binding_stale(record)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build._binding_stale(" ".join(build._binding_command(build._nvcc(), build.BINDING)))
