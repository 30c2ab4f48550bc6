"""Builds libdg.so (the HIP library) in-tree for gfx950 with hipcc."""
from __future__ import annotations

import hashlib
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "libdg.so")
SOURCES = [os.path.join(CSRC, f) for f in ("dg_api.hip", "dg_block.hip")]
DEPS = SOURCES + [os.path.join(CSRC, "marshal.cpp")] + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith(".hpp")] + [
    os.path.join(ROOT, "include", "dg.h")]
# native argument marshalling of the binding: a CPython extension module against torch's headers
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
# measurement companion (streaming-read calibration kernel), loaded by the benchmark only
PROBE_LIB_PATH = os.path.join(PKG, "libdg_probe.so")
PROBE_SOURCES = [os.path.join(CSRC, "hbm_probe.hip")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-shared", "-fPIC",
    # no packed-fp32 VALU instructions (v_pk_*_f32) in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in ordinary VGPRs: the per-K-block promotion reads every partial
    # with VALU FMAs, which cannot take AGPR operands
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    "-Wall", "-Wno-unused-function",
]


def source_hash() -> str:
    """Hash of the sources libdg.so is built from (every csrc file and dg.h): compiled
    into the library as its build id, and compared with the sources by the binding."""
    h = hashlib.sha256()
    for path in sorted(DEPS):
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode() + f.read())
    return h.hexdigest()[:16]


def marshal_command(out: str = MARSHAL_PATH) -> list[str]:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DDG_BUILD_ID="{source_hash()}"',
            *(f"-isystem{d}" for d in (*include_paths(), sysconfig.get_paths()["include"], "/opt/rocm/include")),
            "-o", out, MARSHAL_SOURCE, f"-L{lib}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-ltorch",
            f"-Wl,-rpath,{lib}"]


def _compile(cmd: list[str], what: str, verbose: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln]
    if res.returncode != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"{cmd[0]} failed building {what}")
    if verbose and msgs:
        sys.stderr.write("\n".join(msgs) + "\n")


def build_marshal(verbose: bool = False) -> bool:
    """_marshal.so, which only saves host time: libdg.so needs hipcc alone, so where g++, torch's or
    Python's headers are missing the build goes on and the binding checks arguments in Python."""
    try:
        _compile(marshal_command(), "_marshal.so", verbose)
        return True
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(MARSHAL_PATH):
            os.remove(MARSHAL_PATH)  # of other sources
        sys.stderr.write(f"_marshal.so is not built ({e}): the binding checks arguments in Python\n")
        return False


def build(verbose: bool = False, out: str = LIB_PATH, extra: list[str] | None = None) -> str:
    """Compiles the translation units of libdg.so, the binding's marshalling module and the probe
    library side by side, then links libdg.so."""
    with tempfile.TemporaryDirectory(prefix="dg_build_") as tmp:
        compile_only = [f for f in HIPCC_FLAGS if f != "-shared"]
        units = [(src, os.path.join(tmp, os.path.basename(src) + ".o")) for src in SOURCES]
        jobs = [(["hipcc", *compile_only, f'-DDG_BUILD_ID="{source_hash()}"', *(extra or []), "-c", "-o", obj,
                  src], os.path.basename(src)) for src, obj in units]
        jobs.append((["hipcc", *HIPCC_FLAGS, "-o", PROBE_LIB_PATH, *PROBE_SOURCES], "libdg_probe.so"))
        with ThreadPoolExecutor(len(jobs) + 1) as pool:
            marshal = pool.submit(build_marshal, verbose)
            list(pool.map(lambda job: _compile(*job, verbose), jobs))
            marshal.result()
        _compile(["hipcc", "--offload-arch=gfx950", "-shared", "-fPIC", "-o", out, *(obj for _, obj in units)],
                 "libdg.so", verbose)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
