"""The build's own decisions, with stand-ins for the compilers: what is compiled again, and what one part's failure leaves
of the other."""
import os
import subprocess

import pytest
import torch

from mixture_experts_ffn_moe_gb300 import build, gbmoe


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """An empty output folder, compilers that only record what they were asked for."""
    done = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgbmoe.so"))
    monkeypatch.setattr(build, "STEPS", str(tmp_path / "_step_bindings.so"))
    monkeypatch.setattr(build, "STEPS_TORCH", str(tmp_path / "_build" / "step_bindings.torch"), raising=False)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **kw):
        kind = "link" if "nvcc" in cmd[0] and "-shared" in cmd else "binding" if any("step_bindings" in c for c in cmd) else "object"
        done.append(kind)
        if kind in fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    fails = set()
    monkeypatch.setattr(build.subprocess, "run", run)
    return done, fails


def test_the_library_is_linked_though_the_binding_fails(sandbox):
    done, fails = sandbox
    fails.add("binding")
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.STEPS)
    fails.clear()
    done.clear()
    build.build()  # only the binding is left to do
    assert done == ["binding"] and os.path.exists(build.STEPS)


def test_the_library_needs_no_torch(sandbox, monkeypatch):
    done, _ = sandbox
    monkeypatch.setattr(build, "_torch_version", lambda: None)
    build.build()
    assert os.path.exists(build.LIB) and "binding" not in done
    done.clear()
    build.build()
    assert done == []


def test_nothing_is_built_twice_and_another_torch_builds_the_binding_again(sandbox, monkeypatch):
    done, _ = sandbox
    build.build()
    assert done.count("link") == done.count("binding") == 1
    done.clear()
    build.build()
    assert done == []
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert done == ["binding"] and build.steps_built_against() == "0.0.1"


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    build.build()
    monkeypatch.setattr(gbmoe, "_steps", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built against torch"):
        gbmoe._load_steps()
