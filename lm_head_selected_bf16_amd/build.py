"""Build the HIP library libflp.so in-tree with hipcc for gfx950, and the autograd nodes over
it, _flp_torch.so, with g++.

    python -m lm_head_selected_bf16_amd.build

Numerics flags: -ffp-contract=off (no compiler-chosen FMA contraction, so the
arithmetic of every row is fixed by the source) and no fast-math.  Packed
fp32 instructions are disabled for the device code.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libflp.so")
NODES = os.path.join(PKG, "_flp_torch.so")
SOURCES = ["flp_kernels.hip", "flp_rows.hip", "flp_loss.hip", "flp_embed.hip", "flp_dropout.hip", "flp_norm.hip",
           "flp_rms.hip", "flp_adamw.hip", "flp_gated.hip",
           "flp_probe.hip", "flp_noalloc.hip",
           "flp_api.cpp", "flp_plan.cpp"]


def _hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libflp.so)")


def _git_hash() -> str:
    try:
        out = subprocess.run(["git", "-C", ROOT, "rev-parse", "--short", "HEAD"],
                             capture_output=True, text=True, timeout=10)
        return out.stdout.strip() or "unknown"
    except Exception:  # noqa: BLE001
        return "unknown"


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; that is expected.
    errs = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{errs}")
    if verbose and errs.strip():
        print(errs, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every source (always recompiles, side by side) and link libflp.so. Returns the path."""
    flags = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
             "-ffp-contract=off", "-fno-fast-math",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Wno-unused-function",
             f"-DFLP_GIT_HASH=\"{_git_hash()}\"",
             "-I", os.path.join(ROOT, "include")]
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        outs = [os.path.join(objects, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1, 8)) as pool:
            list(pool.map(lambda so: _run([_hipcc(), *flags, "-c", os.path.join(CSRC, so[0]), "-o", so[1]],
                                          verbose), zip(SOURCES, outs)))
        _run([_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *outs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    build_nodes(verbose)
    return LIB


def build_nodes(verbose: bool = False) -> str:
    """Compile the autograd nodes (host code over the C ABI, with torch's headers) into
    _flp_torch.so.  Returns the path."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    tmp = NODES + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-DTORCH_EXTENSION_NAME=_flp_torch", "-DTORCH_API_INCLUDE_EXTENSION_H",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include")]
    for d in [*include_paths(), sysconfig.get_path("include")]:
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "flp_torch.cpp"), "-o", tmp]
    cmd += [f"-L{d}" for d in library_paths()]
    cmd += ["-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed ({res.returncode}):\n{res.stderr}")
    if verbose and res.stderr.strip():
        print(res.stderr, file=sys.stderr)
    os.replace(tmp, NODES)
    return NODES


if __name__ == "__main__":
    print(build(verbose=True))
