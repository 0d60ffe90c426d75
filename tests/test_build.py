"""Building the feed-forward operators' Python binding, with and without what only it needs."""
import os
import sys

import pytest

import message_allreduce_amd as llar
from message_allreduce_amd import _build, ffn


@pytest.fixture
def binding(tmp_path, monkeypatch):
    path = str(tmp_path / "_llar_py.so")
    monkeypatch.setattr(_build, "BINDING", path)
    return path


@pytest.mark.parametrize("compiler", ["gcc", "/opt/rocm/llvm/bin/clang"])
def test_either_compiler_builds_it(binding, compiler, monkeypatch):
    if _build.shutil.which(compiler) is None:
        pytest.skip("no " + compiler)
    monkeypatch.setattr(_build, "_c_compiler", lambda: compiler)
    assert _build._build_binding() and os.path.getsize(binding) > 0


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_without_them_the_library_stays_usable(binding, missing, monkeypatch, tmp_path, capsys):
    with open(binding, "w") as f:
        f.write("an older one")
    if missing == "headers":
        monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    assert not _build._build_binding()
    assert not os.path.exists(binding)
    assert "not built" in capsys.readouterr().err


def test_a_missing_binding_is_an_error_of_the_operators_alone(monkeypatch):
    llar.lib()
    monkeypatch.setattr(ffn, "_native", None)
    monkeypatch.delattr(llar, "_llar_py", raising=False)
    monkeypatch.setitem(sys.modules, llar.__name__ + "._llar_py", None)
    with pytest.raises(llar.LlarError, match="not built"):
        llar.linear(None, None)
