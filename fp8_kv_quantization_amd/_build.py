"""Builds libkvstore.so in-tree with hipcc for gfx950 (its objects are compiled
side by side), its CPython binding (_kvstore_py, gcc) and the tensor-level
binding of the paged operators (_kvstore_torch, g++ against torch's headers),
both linked against libkvstore.so."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "kvstore.hip")
HEADER = os.path.join(ROOT, "include", "kvstore.h")
LIB = os.path.join(PKG, "libkvstore.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
PY_SRC = os.path.join(PKG, "csrc", "kvstore_py.c")
PY_EXT = os.path.join(PKG, "_kvstore_py" + sysconfig.get_config_var("EXT_SUFFIX"))
TORCH_SRC = os.path.join(PKG, "csrc", "kvstore_torch.cpp")
TORCH_EXT = os.path.join(PKG, "_kvstore_torch" + sysconfig.get_config_var("EXT_SUFFIX"))

FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC", "-shared",
    # packed fp32 VALU forms are kept out of generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def objects() -> list:
    """(source, extra flags, object name) of every object of the library: the
    stores, loads and host side, and the attention kernels once per source
    type and cache format."""
    csrc = os.path.join(PKG, "csrc")
    objs = [(os.path.join(csrc, "libkvstore.hip"), [], "libkvstore.o")]
    for fp16 in (0, 1):
        for fmt in range(4):
            for kind in ("split", "tile"):
                objs.append((os.path.join(csrc, f"attention_{kind}.hip"),
                             [f"-DKVATTN_FP16={fp16}", f"-DKVATTN_FMT={fmt}"],
                             f"attention_{kind}_{fp16}_{fmt}.o"))
    return objs


def command(src: str, out: str, extra=()) -> list:
    return [HIPCC, *[f for f in FLAGS if f != "-shared"], *extra,
            "-I", os.path.join(ROOT, "include"), "-c", src, "-o", out]


def link_command(objs, out: str = LIB) -> list:
    return [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", out]


def binding_command(out: str = PY_EXT) -> list:
    return ["gcc", "-O2", "-std=c11", "-shared", "-fPIC", "-Wall", "-Wextra",
            "-D__HIP_PLATFORM_AMD__", "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(ROCM, "include"),
            PY_SRC, "-L", PKG, "-lkvstore", "-Wl,-rpath,$ORIGIN", "-o", out]


def torch_binding_command(out: str = TORCH_EXT) -> list:
    import importlib.util
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-fvisibility=hidden",
            "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
            "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
            "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(ROCM, "include"), TORCH_SRC, "-L", PKG, "-lkvstore", "-L", lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN", "-o", out]


def _run(cmd, out, what, verbose):
    tmp = out + ".tmp"
    cmd = [tmp if c == out else c for c in cmd]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(verbose: bool = False, out: str = LIB, extra=()) -> str:
    """Compile the HIP library and, for the in-tree library, the two bindings
    (always).  Writes atomically."""
    with tempfile.TemporaryDirectory() as tmp:
        made = [(src, os.path.join(tmp, name), [*flags, *extra]) for src, flags, name in objects()]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda m: _run(command(m[0], m[1], m[2]), m[1], "hipcc", verbose), made))
        _run(link_command([m[1] for m in made], out), out, "hipcc (link)", verbose)
    if out == LIB:
        _run(binding_command(), PY_EXT, "gcc (binding)", verbose)
        _run(torch_binding_command(), TORCH_EXT, "g++ (tensor binding)", verbose)
    return out
