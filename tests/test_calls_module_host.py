"""The binding's extension module: its versions, and calls without it."""
import importlib
import os
import sys
import types

import pytest
import torch

from video_diffusion_hybrid_sparse_b200 import binding as vb
from video_diffusion_hybrid_sparse_b200 import build

NAME = "video_diffusion_hybrid_sparse_b200._calls"
FUNCTIONS = ("linear_fwd", "linear_bwd", "linear_step", "norm_fwd", "norm_bwd")


@pytest.fixture
def fresh(monkeypatch):
    """The binding as before its first call, and the package without the module."""
    vb.library()
    monkeypatch.setattr(vb, "_calls", None)
    monkeypatch.delattr(sys.modules["video_diffusion_hybrid_sparse_b200"], "_calls", raising=False)
    return monkeypatch


def test_module_is_of_this_torch():
    module = importlib.import_module(NAME)
    assert module.torch_version == torch.__version__
    assert all(callable(getattr(module, f)) for f in FUNCTIONS)


@pytest.mark.parametrize("module", [None, types.SimpleNamespace(torch_version="1.0.0")], ids=["missing", "other torch"])
def test_calls_without_the_module(fresh, module):
    """A module that cannot be imported, or of another torch, is left out with one warning; the calls go on."""
    fresh.setitem(sys.modules, NAME, module)
    with pytest.warns(RuntimeWarning, match="extension module"):
        calls = vb._direct()
    assert all(getattr(calls, f)(1, 2, 3) is None for f in FUNCTIONS)
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):  # the binding's own check
        vb.add_rmsnorm_fwd(x)


def test_built_again_for_another_torch(tmp_path, monkeypatch):
    """The module is built again for another torch, whatever the files' times say, and not for the same."""
    made = []

    def run(cmd, **kw):
        made.append(cmd)
        open(build.CALLS, "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_calls()
    build.build_calls()
    assert len(made) == 1
    os.utime(build.CALLS, (2 ** 31, 2 ** 31))
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_calls()
    build.build_calls()
    assert len(made) == 2 and '-DVDN_TORCH="9.9.9"' in made[1]
