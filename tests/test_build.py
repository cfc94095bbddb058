"""build.py: the library needs no torch; the extension module follows torch's version (CPU, nothing compiled)."""
import os
import subprocess
import sys

import pytest

from expert_cache_host_router_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_builds_without_torch(tmp_path):
    """With no torch to import and no module yet, build() makes or finds the library and raises nothing."""
    build.build()
    code = ("import sys; sys.modules['torch'] = None\nfrom expert_cache_host_router_b200 import build\n"
            f"build.BIND = {str(tmp_path / 'module.so')!r}\nprint(build.build())")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("libmoe.so"), r.stderr[-2000:]


@pytest.fixture
def made(tmp_path, monkeypatch):
    """_build_bind into a folder of its own; the compiler only notes its calls."""
    pytest.importorskip("torch")
    out = tmp_path / "_moe_bind.so"
    calls = []

    def compiler(cmd):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
    monkeypatch.setattr(build, "BIND", str(out))
    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    return calls


def test_the_module_is_made_again_for_another_torch(made, monkeypatch):
    import torch
    build._build_bind(False)
    build._build_bind(False)
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    build._build_bind(False)
    build._build_bind(False)
    assert len(made) == 2
    build._build_bind(True)
    assert len(made) == 3


def test_no_module_without_torch_headers(made, monkeypatch):
    import torch.utils.cpp_extension as ext
    monkeypatch.setattr(ext, "include_paths", lambda *a: ["/nonexistent"])
    build._build_bind(True)
    assert not made
