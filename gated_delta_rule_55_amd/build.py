"""Build libkda.so (HIP kernels + C ABI) for gfx950 with hipcc, and the Python
modules _fast.so and _fast_latent.so on top of it, in-tree.  The library takes hipcc
alone; where the modules' tools are missing (g++, the headers of Python and torch) they
are left out, and layer.py and latent.py make every call themselves.

Usage: python -m gated_delta_rule_55_amd.build [-v]
"""
import os
import shutil
import subprocess
import sys
import sysconfig
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libkda.so")
SOURCES = ["kda_abi.cpp", "kda_conv.hip", "kda_decode.hip", "kda_headscan.hip", "kda_latent_abi.cpp",
           "kda_latent_attend.hip", "kda_latent_cache.hip", "kda_latent_prefill.hip", "kda_linear.hip",
           "kda_linear_abi.cpp", "kda_linear_decode.hip", "kda_norm.hip", "kda_norm_abi.cpp",
           "kda_prefill.hip"]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Werror", "-Wno-unused-function",
    # Packed-fp32 instructions are kept out of every kernel (the host pass
    # ignores the feature with a warning).
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


# Per-source flags.  The prefill kernels are latency-bound; LLVM's iterative
# ILP scheduler orders the chunk-local stage's phases better (measured on
# MI355X at 32k tokens x 32 heads: chunk-local 0.661 -> 0.646 ms, the state
# scan 0.583 -> 0.586 ms, the pass 1.251 -> 1.240 ms; results are unchanged, since
# only the instruction order differs).
SOURCE_FLAGS = {
    "kda_prefill.hip": ["-mllvm", "-amdgpu-sched-strategy=iterative-ilp"],
}


# The Python module that marshals the layer calls (csrc/kda_torch.cpp): host code
# against torch's headers, on top of libkda.so.
FAST_OUT = os.path.join(PKG, "_fast.so")
FAST_LATENT_OUT = os.path.join(PKG, "_fast_latent.so")  # the same for latent.py (csrc/kda_latent_torch.cpp)


def _torch_root():
    try:
        import torch
    except ImportError:
        return None
    return os.path.dirname(torch.__file__)


def _fast_missing():
    """What the module cannot be built without and is not here, or ''."""
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    troot = _torch_root()
    if troot is None or not os.path.exists(os.path.join(troot, "include", "torch", "csrc", "autograd",
                                                        "python_variable.h")):
        return "torch's headers"
    return ""


def _fast_command(source="kda_torch.cpp", out=None):
    import torch

    troot = _torch_root()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    include = [f"-I{INCLUDE}"] + [f"-isystem{d}" for d in (
        os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
        os.path.join(rocm, "include"), sysconfig.get_paths()["include"])]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
             "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + include +
            [os.path.join(CSRC, source), "-o", (out or FAST_OUT) + ".tmp",
             f"-L{os.path.join(troot, 'lib')}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python",
             f"-L{PKG}", "-l:libkda.so", "-Wl,-rpath,$ORIGIN"])


def _hipcc():
    p = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
    return p if os.path.exists(p) else "hipcc"


def build_fast(verbose: bool = False):
    """Builds the module on top of the built library; its path, or None where its
    tools are missing (an older one would not fit the library and goes)."""
    missing = _fast_missing()
    if missing:
        print(f"{os.path.basename(FAST_OUT)} not built ({missing} not found): layer calls go through ctypes", flush=True)
        if os.path.exists(FAST_OUT):
            os.remove(FAST_OUT)
        return None
    cmd = _fast_command()
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(FAST_OUT + ".tmp", FAST_OUT)
    return FAST_OUT


def build_fast_latent(verbose: bool = False):
    """build_fast for the module behind latent.py."""
    if _fast_missing():
        if os.path.exists(FAST_LATENT_OUT):
            os.remove(FAST_LATENT_OUT)
        return None
    cmd = _fast_command("kda_latent_torch.cpp", FAST_LATENT_OUT)
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(FAST_LATENT_OUT + ".tmp", FAST_LATENT_OUT)
    return FAST_LATENT_OUT


def build(verbose: bool = False, jobs: int = 4) -> str:
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    t0 = time.time()
    for src in SOURCES:
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".cpp") else []
        cmd = ([_hipcc()] + HIPCC_FLAGS + SOURCE_FLAGS.get(src, []) + lang +
               ["-c", os.path.join(CSRC, src), "-o", obj])
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        while sum(p.poll() is None for _, p in procs) >= jobs:
            time.sleep(0.1)
    failed = False
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # the host pass warns that it does not know the packed-fp32 feature
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if lines:
            print(f"[{src}]\n" + "\n".join(lines), flush=True)
        if p.returncode != 0:
            failed = True
    if failed:
        raise RuntimeError("hipcc failed")
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", OUT + ".tmp"] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(OUT + ".tmp", OUT)
    build_fast(verbose)
    build_fast_latent(verbose)
    if verbose:
        print(f"built {OUT} in {time.time() - t0:.1f}s", flush=True)
    return OUT


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
