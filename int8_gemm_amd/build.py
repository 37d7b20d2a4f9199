"""Build libint8_gemm.so (the HIP kernels and the C ABI) for gfx950, and
rowops_bind.so (the host-only binding of the operators between the GEMMs to
torch tensors), in-tree.

    python -m int8_gemm_amd.build            # build the library
    python -m int8_gemm_amd.build --asm DIR  # also write the gfx950 assembly

Compile flags that the method's bit-exactness depends on:
  -ffp-contract=off                          no multiply-add fusion anywhere
  -fhip-fp32-correctly-rounded-divide-sqrt   '/' is the IEEE division
and, for every HIP source on this target, packed-FP32 instruction
selection is switched off (-Xclang -target-feature -Xclang -packed-fp32-ops).
"""
import argparse
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_NAME = "libint8_gemm.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["api.hip", "quantize.hip", "gemm.hip", "hash.hip", "verify.hip", "norm.hip", "checkpoint.hip",
           "logprob.hip"]
ARCH = "gfx950"
BIND_SOURCE = "rowops_bind.cpp"
BIND_PATH = os.path.join(HERE, "rowops_bind.so")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libint8_gemm.so)")


def common_flags():
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-function", "-Wno-unused-command-line-argument",
        "-I", os.path.join(ROOT, "include"),
    ]


def bind_command(out: str):
    """The host compiler's command for the binding (torch's C++ interface and
    the C ABI's header; the C ABI itself is reached by address)."""
    import torch
    from torch.utils import cpp_extension
    cxx = shutil.which(os.environ.get("CXX", "g++")) or "g++"
    includes = [a for p in (*cpp_extension.include_paths(), sysconfig.get_paths()["include"]) for a in ("-isystem", p)]
    libs = [a for p in cpp_extension.library_paths() for a in ("-L", p)]
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *includes, "-o", out,
            os.path.join(CSRC, BIND_SOURCE), *libs, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build_bind(verbose: bool = False) -> str:
    tmp = BIND_PATH + ".tmp"
    cmd = bind_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"the binding's compiler failed with status {res.returncode}")
    os.replace(tmp, BIND_PATH)
    return BIND_PATH


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with status {res.returncode}")


def build(verbose: bool = False, asm_dir: str = None) -> str:
    cc = hipcc()
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB_PATH + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        out = [os.path.join(objs, os.path.basename(s) + ".o") for s in srcs]
        cmds = [[cc, *common_flags(), "-c", "-o", o, s] for o, s in zip(out, srcs)]
        with ThreadPoolExecutor(min(len(srcs), os.cpu_count() or 1)) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), cmds))
        _run([cc, *common_flags(), "-shared", "-o", tmp, *out], verbose)
    # A kernel template whose host-side instantiation fails leaves its launch
    # stub undefined: the link succeeds, but loading the library would not.
    nm = shutil.which("nm")
    if nm:
        und = subprocess.run([nm, "-D", "--undefined-only", tmp], capture_output=True, text=True).stdout
        stubs = [l.split()[-1] for l in und.splitlines() if "__device_stub__" in l]
        if stubs:
            raise RuntimeError("undefined kernel launch stubs in the built library: " + ", ".join(stubs))
    os.replace(tmp, LIB_PATH)
    build_bind(verbose)
    if asm_dir:
        os.makedirs(asm_dir, exist_ok=True)
        for s in srcs:
            out = os.path.join(asm_dir, os.path.basename(s) + f".{ARCH}.s")
            cmd = [cc, *common_flags(), "--cuda-device-only", "-S", "-o", out, s]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError("hipcc -S failed")
    return LIB_PATH


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--asm", default=None, help="directory for gfx950 assembly listings")
    ap.add_argument("-v", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.v, asm_dir=a.asm))


if __name__ == "__main__":
    main()
