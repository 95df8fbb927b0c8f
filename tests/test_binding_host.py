"""The package with and without the module that passes tensors from C++: made
for this torch and Python it is used; missing, broken or made for others it is
left alone, with a warning, and everything else is as it was."""
import os
import shutil
import subprocess
import sys

import pytest

mod = pytest.importorskip("expert_grouping_dispatch_amd")
PKG = os.path.dirname(mod.LIB_PATH)

USE = """
import warnings
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import expert_grouping_dispatch_amd as mod
import torch
assert mod.moe_create_indices_workspace_bytes(100, 8) > 0
assert mod.moe_error_string(1)
x, f8, s = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 32).to(torch.float8_e4m3fn), torch.zeros(2, 1)
i = torch.zeros(2, dtype=torch.int32)
for call in (lambda: mod.moe_quantize_f8(x, f8, s), lambda: mod.moe_dispatch_f8(x, 1, i, f8, s),
             lambda: mod.moe_expert_matmul(x, i, i, x, x), lambda: mod.moe_expert_matmul_f8(f8, s, i, i, f8, s, x),
             lambda: mod.moe_layer_few(x, i, s, f8, f8, x, f8, s, s), lambda: mod.moe_quantize_i8(x, f8, s)):
    try:
        call()
    except ValueError as e:
        assert "HIP device" in str(e), e
    else:
        raise AssertionError
print("USED" if isinstance(mod._fast, type(torch)) else "LEFT", len(said), *[str(w.message) for w in said])
"""


def _package(tmp_path, fast=None):
    """A copy of the package whose module is the file that `fast` writes, if any; what a program that uses it prints."""
    pkg = tmp_path / "expert_grouping_dispatch_amd"
    pkg.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py"):
            shutil.copy(os.path.join(PKG, name), pkg / name)
    os.symlink(mod.LIB_PATH, pkg / "libmoe_route.so")
    if fast is not None:
        fast(pkg)
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_it_is_built_and_used(tmp_path):
    assert isinstance(mod._fast, type(os)) and os.path.exists(os.path.join(PKG, "_fast.so"))
    assert _package(tmp_path, lambda pkg: shutil.copy(os.path.join(PKG, "_fast.so"), pkg)) == "USED 0"


def test_missing(tmp_path):
    said = _package(tmp_path)
    assert said.startswith("LEFT 1 ") and "_fast is not used" in said


def test_broken(tmp_path):
    said = _package(tmp_path, lambda pkg: (pkg / "_fast.so").write_bytes(b"not a library"))
    assert said.startswith("LEFT 1 ") and "_fast is not used" in said


@pytest.mark.parametrize("text", ["made_for = 'torch 0.1, Python 3.1'", ""])
def test_made_for_others(tmp_path, text):
    said = _package(tmp_path, lambda pkg: (pkg / "_fast.py").write_text(text))
    assert said.startswith("LEFT 1 ") and "_fast is not used" in said


def test_a_build_without_its_headers_ends_well(tmp_path, monkeypatch, capsys):
    """The library and the C program are built and returned; the module of an older build goes."""
    import importlib.util

    spec = importlib.util.spec_from_file_location("build_lib_under_test", os.path.join(PKG, "build_lib.py"))
    build_lib = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build_lib)
    old = tmp_path / "_fast.so"
    old.write_bytes(b"of an older library")
    done = []
    monkeypatch.setattr(build_lib, "FAST", str(old))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build_lib, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build_lib, "sources", lambda: ["one.hip"])
    monkeypatch.setattr(build_lib, "_compile", lambda src: src)
    monkeypatch.setattr(build_lib, "build_c_example", lambda verbose: done.append("C"))
    real = subprocess.run

    def run(cmd, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        (tmp_path / "lib.so.tmp").write_bytes(b"")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build_lib.subprocess, "run", run)
    assert build_lib.build(verbose=False) == str(tmp_path / "lib.so")
    monkeypatch.setattr(build_lib.subprocess, "run", real)
    assert done == ["C"] and not old.exists() and "Python.h" in capsys.readouterr().err
