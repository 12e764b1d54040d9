"""The validation layer of latent attention under AddressSanitizer
and UndefinedBehaviorSanitizer on the CPU: its host sources of the C ABI,
built with g++ and both sanitizers and linked with the library's own kernel
objects, run every check of test_latent_abi_host.py in a child process that
preloads the sanitizer runtimes.  Nothing here touches a GPU."""
import glob
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_55_amd", "csrc")
HOST = ("kda_abi", "kda_linear_abi", "kda_norm_abi", "kda_latent_abi")
KERNELS = [os.path.join(ROOT, "gated_delta_rule_55_amd", "_build", os.path.basename(p)[:-4] + ".o")
           for p in sorted(glob.glob(os.path.join(CSRC, "*.hip")))]
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-g", "-O1"]


def _runtime(name):
    p = subprocess.run(["gcc", f"-print-file-name={name}"], capture_output=True, text=True).stdout.strip()
    return p if os.path.isabs(p) and os.path.exists(p) else None


pytestmark = pytest.mark.skipif(
    not (shutil.which("g++") and _runtime("libasan.so") and _runtime("libubsan.so")
         and all(os.path.exists(o) for o in KERNELS)),
    reason="needs g++ with ASan/UBSan runtimes and the library's objects (build first)")


def test_latent_validation_under_sanitizers(tmp_path):
    objs = []
    for name in HOST:
        objs.append(str(tmp_path / (name + ".o")))
        subprocess.run(["g++", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        f"-I{ROOT}/include", f"-I{CSRC}", *SAN, "-c", os.path.join(CSRC, name + ".cpp"),
                        "-o", objs[-1]], check=True)
    lib = str(tmp_path / "libkda_san.so")
    subprocess.run(["g++", "-shared", *SAN, "-o", lib, *objs, *KERNELS, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib"], check=True)
    script = tmp_path / "child.py"
    script.write_text(f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]
from gated_delta_rule_55_amd import _abi
_abi.LIB_PATH = {lib!r}
import pytest
rc = pytest.main(["-q", "-x", "-p", "no:cacheprovider", {os.path.join(ROOT, 'tests', 'test_latent_abi_host.py')!r}])
print("host checks:", int(rc), flush=True)
sys.exit(int(rc))
""")
    env = dict(os.environ, LD_PRELOAD=f"{_runtime('libasan.so')} {_runtime('libubsan.so')}",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    p = subprocess.run([sys.executable, str(script)], env=env, capture_output=True, text=True, timeout=600)
    out = p.stdout + p.stderr
    assert p.returncode == 0 and "host checks: 0" in out, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out
