"""The package without its quick binding: everything works the Python way, and a binding that cannot be used is as one that
is not there (CPU)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "sparse_attention_fp4_quantize_gb300"
PACKAGE = os.path.join(ROOT, NAME)

# Calls of every function that the binding has, on tensors of the CPU with a stand-in for the library.
CALLS = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import %s as csa2
print([str(w.message) for w in seen if "quick binding" in str(w.message)])
import sys, torch
sys.path.insert(0, %r)
import test_paged_fp4_checks as t
csa2._lib, csa2._on_device, csa2._stream = t._FakeLib(), lambda x: True, lambda s: None
for fn, args in t.BINDINGS:
    getattr(csa2, fn)(**args())
print(csa2._lib.calls == [fn for fn, _ in t.BINDINGS])
csa2._bind(t.REAL)
print(t.REAL.csa2_version())
""" % (NAME, os.path.join(ROOT, "tests"))


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__._build_module().build()


def _package(tmp_path, binding):
    """A copy of the package (by links) with this binding, or none."""
    at = tmp_path / NAME
    at.mkdir()
    for f in os.listdir(PACKAGE):
        if f.endswith(".py") or f == "libcsa2.so":
            os.symlink(os.path.join(PACKAGE, f), at / f)
    if binding is not None:
        (at / "_csa2_bind.so").write_bytes(binding)
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


def _binding():
    with open(os.path.join(PACKAGE, "_csa2_bind.so"), "rb") as f:
        return f.read()


def test_the_package_works_with_its_binding(built, tmp_path):
    assert _package(tmp_path, _binding()) == ["[]", "True", "100"]


@pytest.mark.parametrize("binding", [None, b"", b"no library"])
def test_the_package_works_without_its_binding(built, tmp_path, binding):
    said, called, version = _package(tmp_path, binding)
    assert "quick binding" in said and called == "True" and version == "100"


def test_the_package_leaves_a_binding_for_another_torch_alone(built, tmp_path):
    """at::Tensor's layout is another's there: the binding says what it was built for."""
    import torch
    mine = ("torch %s," % torch.__version__).encode()
    other = mine[:-2] + (b"9" if mine[-2:-1] != b"9" else b"8") + b","
    assert _binding().count(mine) == 1
    said, called, version = _package(tmp_path, _binding().replace(mine, other))
    assert "quick binding" in said and other.decode() in said and called == "True" and version == "100"


def test_the_package_leaves_a_binding_that_says_nothing_alone(built, tmp_path):
    said, called, version = _package(tmp_path, _binding().replace(b"built_for\0", b"built_xyz\0"))
    assert "quick binding" in said and called == "True" and version == "100"


def test_a_binding_for_another_torch_is_built_anew(built, tmp_path, monkeypatch):
    import __graft_entry__
    m = __graft_entry__._build_module()
    assert m.up_to_date()
    monkeypatch.setattr(m, "built_for", lambda: "torch 0.0, another Python")
    assert not m.up_to_date()
    monkeypatch.setattr(m, "BIND", str(tmp_path / "_csa2_bind.so"))
    m._build_bind()
    assert m.up_to_date()
    monkeypatch.undo()
    assert m.up_to_date()


def test_the_library_is_built_without_a_compiler_for_the_binding(built, tmp_path, monkeypatch, capsys):
    """No torch headers, no host compiler: the library is there all the same, and no binding of before is left."""
    import __graft_entry__
    m = __graft_entry__._build_module()
    old = tmp_path / "_csa2_bind.so"
    old.write_bytes(b"of before")
    monkeypatch.setattr(m, "BIND", str(old))
    monkeypatch.setenv("CXX", "false")
    before = os.path.getmtime(m.LIB)
    assert m.build() == m.LIB and os.path.exists(m.LIB)
    assert os.path.getmtime(m.LIB) == before                             # nor is the library compiled again for it
    assert not old.exists() and "_csa2_bind.so" in capsys.readouterr().err
    monkeypatch.delenv("CXX")
    m.build()
    assert old.exists() and m.up_to_date() and os.path.getmtime(m.LIB) == before
    monkeypatch.setattr(m, "_torch", lambda: str(tmp_path))             # no torch
    assert m.build() == m.LIB and not old.exists()
