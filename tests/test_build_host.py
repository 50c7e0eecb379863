"""The build without a compiler at work: the C library needs nvcc alone, whatever becomes of the torch binding."""
import subprocess
import types

import pytest

from min_sampling_gb300 import build


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """Stand-ins for the tools: each call writes its output file; `fails` names a tool that returns an error."""
    state = types.SimpleNamespace(fails=None, calls=[])

    def run(cmd, **kw):
        state.calls.append(cmd[0])
        if state.fails is not None and cmd[0].endswith(state.fails):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "DECODE", str(tmp_path / "_decode.so"))
    state.lib, state.decode = tmp_path / "lib.so", tmp_path / "_decode.so"
    return state


def test_everything_is_built(tools):
    assert build.build() == str(tools.lib)
    assert tools.lib.exists() and tools.decode.exists() and tools.calls.count("g++") == 2


def test_without_torch_the_library_is_built(tools, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == str(tools.lib)
    assert tools.lib.exists() and not tools.decode.exists() and "g++" not in tools.calls


def test_a_binding_that_does_not_compile_leaves_the_library(tools):
    tools.fails = "g++"
    with pytest.raises(RuntimeError, match="decode_binding"):
        build.build()
    assert tools.lib.exists()


def test_a_kernel_that_does_not_compile_fails(tools):
    tools.fails = "nvcc"
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    assert not tools.lib.exists()
