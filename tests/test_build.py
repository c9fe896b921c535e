"""What the build makes, from which sources, and when: the commands are recorded
and stand for the files they would make."""
import os
import sys

import pytest

from microscaled_precision_moe_gb300 import build as B


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The commands run, in a package folder of its own with the real sources."""
    ran = []

    def run(cmd, what, verbose=False):
        ran.append((what, cmd))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "nvcc", lambda: "nvcc")
    for name, path in (("BUILD", "_build"), ("LIB", "libmpm.so"), ("BINDING", "_binding.so"),
                       ("BINDING_FOR", "_build/binding_for.txt")):
        monkeypatch.setattr(B, name, str(tmp_path / path))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    return ran


def _without_torch(monkeypatch):
    for name in [m for m in sys.modules if m == "torch" or m.startswith("torch.")]:
        monkeypatch.delitem(sys.modules, name)
    monkeypatch.setitem(sys.modules, "torch", None)        # import torch: ImportError


def test_library_and_binding(made):
    assert B.needs_build() and B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING)
    order = [w for w, _ in made]
    assert order.index("link of libmpm.so") < order.index("link of _binding.so")
    n = len(made)
    assert not B.needs_build() and B.build() == B.LIB and len(made) == n


def test_the_library_alone_without_torch(made, monkeypatch):
    _without_torch(monkeypatch)
    assert B.needs_build() and B.build(force=True) == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    assert all(cmd[0] == "nvcc" for _, cmd in made)
    assert not B.needs_build() and B.build() == B.LIB


def test_a_binding_that_fails_leaves_the_library(made, monkeypatch):
    run = B._run

    def fails(cmd, what, verbose=False):
        if cmd[0] == "g++":
            raise RuntimeError(f"{what} failed")
        run(cmd, what, verbose)

    monkeypatch.setattr(B, "_run", fails)
    with pytest.raises(RuntimeError, match="binding.cpp failed"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_only_what_is_out_of_date(made, tmp_path, monkeypatch):
    B.build()
    made.clear()
    source = tmp_path / "binding.cpp"
    source.write_text("")
    future = os.path.getmtime(B.BINDING) + 10
    os.utime(source, (future, future))
    monkeypatch.setattr(B, "BINDING_SRC", str(source))
    B.build()
    assert {cmd[0] for _, cmd in made} == {"g++"}


def test_another_torch_rebuilds_the_binding(made, monkeypatch):
    import torch
    B.build()
    made.clear()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert B.needs_build()
    B.build()
    assert {cmd[0] for _, cmd in made} == {"g++"} and not B.needs_build()
    assert any("torch 9.9.9" in arg for _, cmd in made for arg in cmd)


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    import torch
    from microscaled_precision_moe_gb300 import _lib, ops
    B.build()
    monkeypatch.setattr(ops, "_native_module", None)
    assert ops._native().built_for == _lib.binding_abi()
    monkeypatch.setattr(ops, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(_lib.MpmError, match="built for torch .* this is torch 9.9.9"):
        ops._native()
