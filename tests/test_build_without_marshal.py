"""CPU: libdg.so is built and used where the native marshalling module cannot be (no g++, no headers):
the build goes on, and the binding's Python checks make the calls."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "fp8_block_scaled_dg_amd")


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """build.py as a module, with its outputs in tmp_path and its compilations recorded."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    mod.made, mod.failing = [], None

    def compile_(cmd, what, verbose):
        if what == "_marshal.so" and mod.failing:
            raise mod.failing
        mod.made.append(what)

    monkeypatch.setattr(mod, "_compile", compile_)
    return mod


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), RuntimeError("g++ failed building _marshal.so"),
                                   ImportError("No module named 'torch'")])
def test_the_build_goes_on(builder, error, tmp_path, capsys):
    (tmp_path / "_marshal.so").write_bytes(b"of other sources")
    builder.failing = error
    assert builder.build(out=str(tmp_path / "libdg.so")) == str(tmp_path / "libdg.so")
    assert builder.made[-1] == "libdg.so" and "dg_block.hip" in builder.made
    assert not (tmp_path / "_marshal.so").exists() and "_marshal.so is not built" in capsys.readouterr().err


def test_a_whole_build_has_both(builder, tmp_path):
    builder.build(out=str(tmp_path / "libdg.so"))
    assert {"_marshal.so", "libdg.so", "libdg_probe.so", "dg_api.hip", "dg_block.hip"} == set(builder.made)


def test_a_failed_library_fails_the_build(builder, monkeypatch, tmp_path):
    def compile_(cmd, what, verbose):
        if what == "dg_block.hip":
            raise RuntimeError("hipcc failed building dg_block.hip")

    monkeypatch.setattr(builder, "_compile", compile_)
    with pytest.raises(RuntimeError, match="dg_block"):
        builder.build(out=str(tmp_path / "libdg.so"))


def test_the_binding_without_the_module(tmp_path):
    for name in ("__init__.py", "libdg.so"):
        os.makedirs(tmp_path / "fp8_block_scaled_dg_amd", exist_ok=True)
        shutil.copy(os.path.join(PKG, name), tmp_path / "fp8_block_scaled_dg_amd" / name)
    shutil.copy(os.path.join(PKG, "build.py"), tmp_path / "fp8_block_scaled_dg_amd" / "build.py")
    shutil.copytree(os.path.join(PKG, "csrc"), tmp_path / "fp8_block_scaled_dg_amd" / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    code = ("import torch, fp8_block_scaled_dg_amd as m\n"
            "assert not hasattr(m._marshal, 'bind')\n"
            "x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)\n"
            "for call in (lambda: m.layernorm_fp8_1x128(x, w), lambda: m.layernorm_backward(x, x, w, w, w),\n"
            "             lambda: m.dropout_add(x, 0.1, None), lambda: m.dropout_backward_fp8(x, 0.1, None),\n"
            "             lambda: m.gated_backward_fp8(x, x),\n"
            "             lambda: m.fp8_gemm_nt_gated_fp8(x.view(torch.uint8), x.view(torch.uint8), w, w)):\n"
            "    try:\n"
            "        call()\n"
            "    except ValueError as e:\n"
            "        assert 'GPU tensor' in str(e), e\n"
            "    else:\n"
            "        raise AssertionError('not refused')\n"
            "print('refused all')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused all" in r.stdout, r.stderr
