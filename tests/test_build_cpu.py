"""The build of the Python module: rebuilt for another torch, left alone otherwise."""
import os

import torch

import sparse_mixture_experts_smoe_b200 as smoe
from sparse_mixture_experts_smoe_b200 import build


def _paths(monkeypatch, tmp_path, stamp, module=True):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "binding.txt"))
    if module:
        (tmp_path / "_binding.so").write_text("built")
    if stamp is not None:
        (tmp_path / "binding.txt").write_text(stamp)
    calls = []

    def run(cmd, check):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("rebuilt")

    monkeypatch.setattr(build.subprocess, "run", run)
    return calls


def test_module_for_another_torch_is_rebuilt(monkeypatch, tmp_path):
    calls = _paths(monkeypatch, tmp_path, "torch 0.0, cpython-0")
    assert build.binding_stale()
    build._build_binding(False)
    assert len(calls) == 1 and (tmp_path / "_binding.so").read_text() == "rebuilt"
    assert torch.__version__ in (tmp_path / "binding.txt").read_text()
    assert not build.binding_stale()
    build._build_binding(False)
    assert len(calls) == 1


def test_module_without_a_record_is_rebuilt_by_a_build_only(monkeypatch, tmp_path):
    calls = _paths(monkeypatch, tmp_path, None)
    assert not build.binding_stale()
    build._build_binding(False)
    assert len(calls) == 1


def test_first_call_builds_a_stale_module(monkeypatch):
    built = []
    monkeypatch.setattr(smoe, "_native", None)
    monkeypatch.setattr(build, "binding_stale", lambda: True)
    monkeypatch.setattr(build, "build", lambda: built.append(1))
    smoe._calls()
    assert built == [1]


def test_module_is_built_for_this_torch():
    smoe._calls()
    assert os.path.exists(build.BINDING) and not build.binding_stale()
