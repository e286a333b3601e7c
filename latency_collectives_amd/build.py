"""Build the HIP library (libar.so) for gfx950 in-tree, and the bindings of the decode and the serving operators.

    python -m latency_collectives_amd.build

compiles every ``csrc/*.hip`` (collectives), ``csrc_decode/*.hip`` (decode operators) and
``csrc_serving/*.hip`` (serving operators) file with hipcc into ``latency_collectives_amd/libar.so``, and
``csrc_decode/ar_decode_bind.cpp`` and ``csrc_serving/ar_serving_bind.cpp`` (host code against torch's headers)
with the C++ compiler into ``_decode_calls.so`` and ``_serving_calls.so`` beside it.
"""

from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_DECODE = os.path.join(PKG, "csrc_decode")
CSRC_SERVING = os.path.join(PKG, "csrc_serving")
LIB = os.path.join(PKG, "libar.so")
CALLS = os.path.join(PKG, "_decode_calls.so")
SERVING_CALLS = os.path.join(PKG, "_serving_calls.so")
ARCH = os.environ.get("AR_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # Never let the compiler form packed fp32 instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def sources() -> list[str]:
    return sorted(f for d in (CSRC, CSRC_DECODE, CSRC_SERVING)
                  for f in glob.glob(os.path.join(d, "*.hip")))


def build(verbose: bool = False) -> str:
    """Compile the library unconditionally and return its path. Every source is compiled to an
    object file in its own hipcc process (in parallel), then the objects are linked."""
    import tempfile
    from concurrent.futures import ThreadPoolExecutor

    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp"
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="ar_build_") as d:
        objs = [os.path.join(d, os.path.basename(src) + ".o") for src in sources()]
        cmds = [[hipcc, *compile_flags, "-c", src, "-o", obj]
                for src, obj in zip(sources(), objs)]
        cmds.append([hipcc, *HIPCC_FLAGS, *objs, "-o", tmp])

        def run(cmd):
            if verbose:
                print(" ".join(cmd), flush=True)
            return subprocess.run(cmd, capture_output=True, text=True)

        with ThreadPoolExecutor(max_workers=len(objs)) as pool:
            results = list(pool.map(run, cmds[:-1]))
        results.append(run(cmds[-1]) if all(r.returncode == 0 for r in results) else None)
        for r in results:
            if r is None or r.returncode != 0:
                for q in results:
                    if q is not None:
                        sys.stderr.write(q.stdout + q.stderr)
                raise RuntimeError("hipcc failed to build libar.so")
    os.replace(tmp, LIB)
    build_calls(verbose)
    return LIB


def build_calls(verbose: bool = False) -> None:
    """Compile the bindings (libar.so must be there), side by side."""
    import sysconfig
    from concurrent.futures import ThreadPoolExecutor

    import torch

    root = os.path.dirname(torch.__file__)

    def compile(source, target):
        # -D: what the HIP headers and torch's ask of a plain C++ compiler
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
               "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
               "-I", os.path.join(root, "include"),
               "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-I", "/opt/rocm/include", "-I", sysconfig.get_paths()["include"],
               source, "-o", target + ".tmp", "-L", PKG, "-lar",
               "-L", os.path.join(root, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python",
               "-Wl,-rpath,$ORIGIN"]
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.run(cmd, capture_output=True, text=True)

    jobs = [(os.path.join(CSRC_DECODE, "ar_decode_bind.cpp"), CALLS),
            (os.path.join(CSRC_SERVING, "ar_serving_bind.cpp"), SERVING_CALLS)]
    with ThreadPoolExecutor(max_workers=len(jobs)) as pool:
        results = list(pool.map(lambda j: compile(*j), jobs))
    for (_, target), r in zip(jobs, results):
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"the C++ compiler failed to build {os.path.basename(target)}")
        os.replace(target + ".tmp", target)


def ensure_built() -> str:
    """Build only what does not exist yet (tests and tools call this)."""
    if not os.path.exists(LIB):
        build()
    elif not (os.path.exists(CALLS) and os.path.exists(SERVING_CALLS)):
        build_calls()
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
