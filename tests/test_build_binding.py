"""When the compiled binding is built: beside the library, and by itself where it is missing or
was built against another torch.  The compilers are stand-ins."""

from __future__ import annotations

import importlib

import pytest

import attention_flashattention_fwd_03_gb300 as gb
from attention_flashattention_fwd_03_gb300 import build

torch = pytest.importorskip("torch")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree whose library is newer than its sources; `built` counts builds of _binding."""
    lib = tmp_path / "lib.so"
    lib.write_text("")
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "_build" / "stamp"))
    tree = type("Tree", (), dict(path=tmp_path, built=0, wrong=None))

    def fake():
        tree.built += 1
        if tree.wrong is None:
            (tmp_path / "_binding.so").write_text("")
        return tree.wrong

    monkeypatch.setattr(build, "build_binding", fake)
    return tree


def test_a_missing_binding_is_built_once(tree):
    for _ in range(2):
        build.build()
        assert tree.built == 1
    (tree.path / "_binding.so").unlink()
    build.build()
    build.build()
    assert tree.built == 2


def test_another_torch_needs_another_binding(tree, monkeypatch):
    build.build()
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1+other")
    build.build()
    build.build()
    assert tree.built == 2


def test_a_failure_is_not_repeated_and_named(tree, capsys, monkeypatch):
    tree.wrong = "no such compiler"
    build.build()
    assert "no such compiler" in capsys.readouterr().err
    build.build()
    assert tree.built == 1 and capsys.readouterr().err == ""
    tree.wrong = None
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1+other")
    build.build()
    assert tree.built == 2 and (tree.path / "_binding.so").exists()


def test_without_torch_there_is_nothing_to_build(tree, monkeypatch):
    monkeypatch.setattr(build, "torch_version", lambda: None)
    build.build()
    assert tree.built == 0


def test_a_tree_that_cannot_be_written_to_is_left_alone(tree, monkeypatch):
    monkeypatch.setattr(build.os, "access", lambda path, mode: False)
    build.build()
    assert tree.built == 0


def test_the_version_is_the_installed_torchs(monkeypatch):
    assert build.torch_version() == torch.__version__
    modules = {n: m for n, m in build.sys.modules.items() if n != "torch"}
    monkeypatch.setattr(build, "sys", type("Sys", (), dict(modules=modules)))
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name: type("Spec", (), dict(origin=torch.__file__)))
    assert build.torch_version() == torch.__version__


def test_calls_without_the_binding_say_so(monkeypatch):
    if not hasattr(torch._C, "_cuda_getDevice"):
        pytest.skip("a torch without CUDA has no quick way")
    gb.lib()

    def missing(name, package=None):
        raise ImportError("no module named _binding")

    monkeypatch.setattr(importlib, "import_module", missing)
    monkeypatch.setattr(gb, "_quick", None)
    with pytest.warns(RuntimeWarning, match="_binding cannot be used"):
        gb._load_quick(torch)
    assert gb._quick is None
