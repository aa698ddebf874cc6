"""When the compiled Python entry points of the layer operators are built anew (no compiler runs here)."""
import os
import subprocess

import pytest

from selective_state_space_mamba_gb300 import _build


@pytest.fixture
def builds(tmp_path, monkeypatch):
    """The commands that build_binding runs; each makes its output."""
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    if hasattr(_build, "BINDING_KEY"):
        monkeypatch.setattr(_build, "BINDING_KEY", str(tmp_path / "_build" / "binding.key"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(str(len(ran)))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build.subprocess, "run", run)
    return ran


def test_once_for_the_same_torch_and_python(builds):
    assert _build.build_binding() == _build.BINDING and len(builds) == 1
    _build.build_binding()
    assert len(builds) == 1
    _build.build_binding(force=True)
    assert len(builds) == 2
    os.utime(_build.BINDING, (0, 0))  # older than its source
    _build.build_binding()
    assert len(builds) == 3


def test_again_for_another_torch_python_or_command(builds, monkeypatch):
    import sysconfig
    import torch
    _build.build_binding()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        _build.build_binding()
        assert len(builds) == 2
        _build.build_binding()
        assert len(builds) == 2
    _build.build_binding()
    assert len(builds) == 3
    with monkeypatch.context() as m:
        real = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda n: ".other.so" if n == "EXT_SUFFIX" else real(n))
        _build.build_binding()
        assert len(builds) == 4
    _build.build_binding()
    with monkeypatch.context() as m:
        m.setattr(_build, "CSRC", os.path.join(_build.CSRC, "."))  # another command
        _build.build_binding()
    assert len(builds) == 6


def test_a_module_without_a_key_is_not_trusted(builds):
    """As one that was built before there was a key, or whose build was interrupted."""
    with open(_build.BINDING, "w") as f:
        f.write("of unknown origin")
    _build.build_binding()
    assert len(builds) == 1


def test_a_current_module_needs_no_compiler(builds, monkeypatch):
    _build.build_binding()
    monkeypatch.setattr(_build, "nvcc", lambda: pytest.fail("looked for"))
    _build.build_binding()
    assert len(builds) == 1
