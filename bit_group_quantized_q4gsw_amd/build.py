"""Build the q4gsw HIP library (libq4gsw.so) in-tree for gfx950.

Each csrc/*.hip file is compiled by hipcc in parallel and the objects are linked
into bit_group_quantized_q4gsw_amd/libq4gsw.so.  Every compile passes
-Xclang -target-feature -Xclang -packed-fp32-ops so no packed-fp32 VALU
instruction is generated.  csrc/host.cpp, the marshalling of torch tensors for the serving
calls, becomes the module _host (_host.so) beside it, by the host compiler; where there is no torch or
no host compiler it is left out, and the binding marshals those calls in Python.
"""
import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libq4gsw.so")
HOST = os.path.join(HERE, "_host.so")
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = os.environ.get("Q4GSW_ARCH", "gfx950")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

CFLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-4] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if noise not in l]
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), flush=True)
    return obj


def _host(verbose: bool) -> None:
    spec = importlib.util.find_spec("torch")
    cxx = shutil.which("g++") or shutil.which("c++")
    if spec is None or spec.origin is None or cxx is None:
        if os.path.exists(HOST):                     # of another environment
            os.remove(HOST)
        print(f"{HOST} is left out: " + ("no host compiler" if cxx is None else "no torch"), file=sys.stderr, flush=True)
        return
    torch = os.path.dirname(spec.origin)
    tmp = HOST + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "host.cpp"), "-o", tmp,
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("the host compiler failed for host.cpp:\n" + res.stdout + res.stderr)
    os.replace(tmp, HOST)


def build(verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    jobs = jobs or min(len(srcs), max(1, min(8, os.cpu_count() or 1)))
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        host = ex.submit(_host, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        tmp = LIB + ".tmp"
        cmd = [HIPCC, "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True, capture_output=not verbose)
        os.replace(tmp, LIB)
        host.result()                                # the library is there whatever becomes of _host
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
