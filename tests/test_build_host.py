"""The build of the two shared objects, with the compilers faked: what is built
when, and what is left when one of them fails. No GPU."""
import os
import subprocess

import pytest

from rope_period_truncated_b200 import build as wpbuild


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Build into an empty folder; returns the list of what was compiled, and the programs that are missing."""
    monkeypatch.setattr(wpbuild, "LIB", str(tmp_path / "libwaveprune.so"))
    monkeypatch.setattr(wpbuild, "BINDING", str(tmp_path / "_calls.so"))
    built, missing = [], set()

    def call(cmd, **_):
        name = os.path.basename(cmd[0])
        if name in missing:
            raise FileNotFoundError(name)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(name)
        built.append(name)

    monkeypatch.setattr(subprocess, "check_call", call)
    return built, missing


def test_library_is_built_where_the_binding_cannot_be(compilers):
    built, missing = compilers
    missing.add("g++")
    with pytest.raises(FileNotFoundError):
        wpbuild.build()
    assert built == ["nvcc"] and os.path.exists(wpbuild.LIB) and not os.path.exists(wpbuild.BINDING)
    missing.clear()
    wpbuild.build()
    assert built == ["nvcc", "g++"] and os.path.exists(wpbuild.BINDING)
    wpbuild.build()
    assert built == ["nvcc", "g++"]  # nothing has changed


def test_binding_of_another_torch_or_python_is_rebuilt(compilers, monkeypatch):
    import sysconfig

    import torch
    built, _ = compilers
    wpbuild.build()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    wpbuild.build()
    assert built == ["nvcc", "g++", "g++"]
    was = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else was(name))
    wpbuild.build()
    wpbuild.build()
    assert built == ["nvcc"] + 3 * ["g++"]


def test_binding_of_unknown_origin_is_rebuilt(compilers):
    built, _ = compilers
    for path in (wpbuild.LIB, wpbuild.BINDING):
        open(path, "w").close()
    wpbuild.build()
    assert built == ["g++"]


def test_import_errors_say_what_is_wrong(monkeypatch, tmp_path):
    """A binding that is not there is to be built; one that does not load says why."""
    import sys

    import rope_period_truncated_b200 as wp
    from rope_period_truncated_b200 import serving

    monkeypatch.setitem(sys.modules, "rope_period_truncated_b200._calls", None)  # the import fails
    monkeypatch.delattr(wp, "_calls", raising=False)
    monkeypatch.setattr(wpbuild, "BINDING", str(tmp_path / "_calls.so"))
    with pytest.raises(ImportError, match="not built"):
        serving._Native().rope_qk
    open(wpbuild.BINDING, "w").close()
    with pytest.raises(ImportError, match="does not load.*_calls") as e:
        serving._Native().rope_qk
    assert "not built" not in str(e.value) and isinstance(e.value.__cause__, ImportError)
