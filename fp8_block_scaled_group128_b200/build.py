"""Build libfp8bs.so (the CUDA kernels and the C ABI) in-tree for sm_100a, and
_decode.so (the native Python binding of its decode calls, linked against it).

    python -m fp8_block_scaled_group128_b200.build [--force]

Each .cu file under csrc/ is compiled by nvcc in parallel to an object file
under _build/, then linked into ``libfp8bs.so`` next to this file;
csrc/decode_binding.cpp is compiled by g++ against the installed torch. Both
are rebuilt whenever the SHA-256 of the sources, headers, this script, the
compiler flags and the torch and Python versions differs from the one recorded
beside them (``libfp8bs.so.stamp``); file times play no part, so a library copied to
another machine with its sources is reused only if it was built from exactly
those sources.
"""

import argparse
import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8bs.so")
STAMP = LIB + ".stamp"
DECODE = os.path.join(PKG, "_decode.so")
DECODE_SRC = os.path.join(CSRC, "decode_binding.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", os.path.join(ROOT, "include")]


def nvcc():
    cand = [os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"),
            shutil.which("nvcc") or ""]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [DECODE_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__])


def source_digest():
    """SHA-256 over every source and header (by name and content), this
    script and the compiler flags."""
    h = hashlib.sha256()
    for d in sorted(_deps()):
        h.update(os.path.relpath(d, ROOT).encode() + b"\0")
        with open(d, "rb") as f:
            h.update(f.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    h.update(f"{torch.__version__} {sys.version_info[:2]}".encode())
    return h.hexdigest()


def up_to_date():
    if not all(os.path.exists(p) for p in (LIB, DECODE, STAMP)):
        return False
    with open(STAMP) as f:
        return f.read().strip() == source_digest()


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc()] + ARCH + FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r.returncode, r.stdout + r.stderr


def _decode_command(out):
    """g++ for the native binding; torch's and CUDA's headers, this library."""
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in include:
        cmd += ["-isystem" if d != include[0] else "-I", d]
    return cmd + [DECODE_SRC, "-o", out, "-L", PKG, "-l:" + os.path.basename(LIB), "-L",
                  os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                  "-Wl,-rpath,$ORIGIN"]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{what} failed")


def build(force=False, verbose=False):
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        for src, obj, rc, log in ex.map(_compile, _sources()):
            if verbose or rc != 0:
                sys.stderr.write(f"--- {os.path.basename(src)}\n{log}")
            if rc != 0:
                raise RuntimeError(f"nvcc failed on {src}")
            objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    _run(cmd, "link")
    os.replace(tmp, LIB)
    tmp = DECODE + ".tmp"
    _run(_decode_command(tmp), "compiling the native binding")
    os.replace(tmp, DECODE)
    with open(STAMP, "w") as f:
        f.write(source_digest() + "\n")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
