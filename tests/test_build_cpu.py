"""The build's two products: libortho.so needs nothing that the Python binding needs."""

import os

import pytest

from orthonormal_optimizer_update_amd import build


@pytest.fixture
def linked(monkeypatch, tmp_path):
    """What a build with stand-ins for the compilers linked, in a folder of its own."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libortho.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "_compile", lambda src: src)
    monkeypatch.setattr(build, "_compile_binding", lambda: "binding.o")
    made = []

    def run(what, cmd):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).replace(".tmp", ""))
        with open(out, "w"):
            pass

    monkeypatch.setattr(build, "_run", run)
    return made


def test_both(linked):
    build.build(verbose=False)
    assert linked == ["libortho.so", "_binding.so"] and os.path.exists(build.LIB) and os.path.exists(build.BINDING)


@pytest.mark.parametrize("error", [RuntimeError("no such header"), ImportError("no torch"), FileNotFoundError("g++")])
def test_the_library_without_the_binding(linked, monkeypatch, error):
    with open(build.BINDING, "w"):   # an older build's, which may not fit the new library
        pass

    def fails():
        raise error

    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="binding") as e:
        build.build(verbose=False)
    assert str(error) in str(e.value) and e.value.__cause__ is error
    assert linked == ["libortho.so"] and os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_no_binding_without_the_library(linked, monkeypatch):
    def fails(src):
        raise RuntimeError(src)

    monkeypatch.setattr(build, "_compile", fails)
    with pytest.raises(RuntimeError):
        build.build(verbose=False)
    assert linked == []
