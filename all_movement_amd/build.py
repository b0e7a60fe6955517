"""Build the HIP library liba2av.so in-tree for gfx950.

Compiles the C ABI runtime, the host planning code and the kernels with hipcc,
each source by itself and side by side, into ``all_movement_amd/liba2av.so``.
Every call recompiles.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "liba2av.so")
SOURCES = ["runtime.hip", "kernels.hip", "plan.cpp", "probe.hip", "moe_host.hip", "moe_gemm.hip",
           "moe_fp8.hip", "moe_route.hip", "moe_rows.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wextra", "-Werror", "-Wno-unused-command-line-argument",
    # Packed-FP32 instructions stay off.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature.
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{out}")
    if verbose and out:
        print(out)


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    compile_flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as objs:
        out = [os.path.join(objs, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=4) as pool:
            list(pool.map(lambda so: _run([HIPCC] + compile_flags +
                                          ["-c", os.path.join(CSRC, so[0]), "-o", so[1]], verbose),
                          zip(SOURCES, out)))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + out + ["-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
