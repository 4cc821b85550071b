"""Builds libskgemm.so in-tree with hipcc for gfx950 (no GPU needed)."""

from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libskgemm.so")
# device-ceiling probes for the roofline (bench.py --ceiling), a library of their own
PROBE_LIB = os.path.join(HERE, "libskprobe.so")
PROBE_SOURCES = ["sk_probe.hip"]
# the native binding of the block-scaled, norm and expert calls: host code against torch's headers
NATIVE = os.path.join(HERE, "_sknative.so")
NATIVE_SOURCES = ["sk_native.cpp", "sk_native_experts.cpp"]
CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["sk_kernels.hip", "sk_kernels_mx.hip", "sk_kernels_ksplit.hip", "sk_backward.hip", "sk_quantize.hip",
           "sk_gemm_block.hip", "sk_norm.hip", "sk_experts.hip", "sk_grouped.hip", "sk_grouped_f16.hip", "sk_rows.hip",
           "sk_quantize4.hip", "sk_api.cpp", "sk_api_block.cpp", "sk_api_experts.cpp"]
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # keep hipcc from emitting packed-fp32 arithmetic on its own
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def build(verbose: bool = False) -> str:
    """Compile every source (in parallel) and link the shared libraries; returns the GEMM library's path.  Where the
    native binding cannot be built, that is said on stderr and only the calls that use it are missing."""
    from concurrent.futures import ThreadPoolExecutor
    objs, cmds = [], []
    for src in SOURCES + PROBE_SOURCES:
        obj = os.path.join(CSRC, os.path.splitext(src)[0] + ".o")
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd.insert(1, "-x")
            cmd.insert(2, "hip")
        cmds.append(cmd)
        objs.append(obj)
    if os.path.exists(NATIVE):
        os.remove(NATIVE)     # (one of another version must not serve this one's library)
    with ThreadPoolExecutor(max_workers=5) as ex:
        native = ex.submit(_build_native, verbose)
        for f in [ex.submit(_run, c, verbose) for c in cmds]:
            f.result()
        n = len(SOURCES)
        for lib, lib_objs in ((LIB, objs[:n]), (PROBE_LIB, objs[n:])):
            tmp = lib + ".tmp"
            _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *lib_objs, "-o", tmp], verbose)
            os.replace(tmp, lib)
        try:
            native.result()
        except (ImportError, OSError, RuntimeError) as e:
            print(f"the native binding was not built (the block-scaled, norm and expert calls of the Python package need it): {e}",
                  file=sys.stderr)
    return LIB


def _build_native(verbose):
    """The native binding, which needs torch and a host compiler; the libraries need neither."""
    _run(_native_command(NATIVE + ".tmp"), verbose)
    os.replace(NATIVE + ".tmp", NATIVE)


def _native_command(out):
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    root = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + sysconfig.get_paths()["include"]]
    for p in include_paths():
        cmd += ["-isystem", p]
    return cmd + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(os.path.join(CSRC, n) for n in NATIVE_SOURCES),
                  "-o", out, "-L" + root, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"build failed: {' '.join(cmd)}\n{out}")
    if verbose and out:
        print(out)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
