"""Build the HIP library libtpl.so in-tree for gfx950 (hipcc cross-compiles; no GPU needed)."""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtpl.so")
# One translation unit per kernel family, compiled in parallel.
SOURCES = ["planner.cpp", "kernels.hip", "kernels_stream.hip", "kernels_quad.hip", "kernels_lds.hip",
           "kernels_lds_w12.hip", "kernels_lds_w48.hip", "kernels_lds_w16.hip",
           "kernels_swap.hip", "kernels_rec.hip", "kernels_etile.hip", "staged.hip",
           "kv_append.hip", "kv_attend.hip", "kv_few.hip", "kv_tile.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wshadow", "-Wno-unused-function",
    # keep the compiler from emitting packed fp32 math
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops"
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if noise not in l and l.strip()]
    if res.returncode != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode})")
    if verbose and msgs:
        print("\n".join(msgs))


# A plain C++ client of the C ABI used by the tests (host code only, links the library).
CLIENT_SRC = os.path.join(ROOT, "tests", "c_abi", "abi_client.cpp")
CLIENT = os.path.join(ROOT, "tests", "c_abi", "abi_client")


# The reading of torch tensors for kv.py: a Python extension (host code only).
CALL_SRC = os.path.join(CSRC, "kv_binding.cpp")
CALL = os.path.join(HERE, "_kv_call.so")


def _call_command(out):
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-isystem", os.path.join(base, "include"), "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
            "-isystem", sysconfig.get_paths()["include"], CALL_SRC, "-o", out,
            "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False) -> str:
    """Build libtpl.so, the binding's extension and the C ABI test client (all in-tree).

    Every source is compiled to an object on its own (in parallel), then the
    objects are linked."""
    compile_flags = [f for f in FLAGS if f != "-shared"]
    objdir = tempfile.mkdtemp(prefix="tpl_build_")
    try:
        objs = [os.path.join(objdir, s + ".o") for s in SOURCES]
        calltmp = CALL + ".tmp"
        jobs = [_call_command(calltmp)]
        jobs += [[HIPCC] + compile_flags + ["-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]
        workers = max(1, min(len(jobs), os.cpu_count() or 1, 16))
        with cf.ThreadPoolExecutor(max_workers=workers) as ex:
            for f in [ex.submit(_run, j, verbose) for j in jobs]:
                f.result()
        tmp = LIB + ".tmp"
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp], verbose)
        os.replace(tmp, LIB)
        os.replace(calltmp, CALL)
    finally:
        shutil.rmtree(objdir, ignore_errors=True)
    if os.path.exists(CLIENT_SRC):
        ctmp = CLIENT + ".tmp"
        _run([HIPCC, "-O2", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "include"), CLIENT_SRC,
              "-L", HERE, "-ltpl", "-Wl,-rpath,$ORIGIN/../../tensor_layout_amd", "-o", ctmp], verbose)
        os.replace(ctmp, CLIENT)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
