"""The launches of linear attention and the norms without a GPU: the library
over stand-ins for the HIP runtime's launch calls (fake_hip.cpp), in a child
process that preloads them.  Which kernels a descriptor enqueues, and what
becomes of a launch's status."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not (shutil.which("g++") and os.path.exists(os.path.join(ROOT, "gated_delta_rule_55_amd", "libkda.so"))),
    reason="needs g++ and libkda.so")

CHILD = """
import ctypes, sys
sys.path[:0] = [{root!r}]
from gated_delta_rule_55_amd import _abi, _abi_layer as al
fake = ctypes.CDLL({fake!r})
fake.fake_log.restype = ctypes.c_char_p
L = al.lib()

def prefill_desc(**over):
    kw = dict(dtype=2, n_seqs=1, n_heads=32, dk=128, dv=128, t_total=300, q=1 << 40, k=2 << 40, v=3 << 40,
              g=4 << 40, o=5 << 40, h0=6 << 40, ht=6 << 40, cu_seqlens=7 << 40)
    kw.update(over)
    return al.make(al.LinearPrefillDesc, **kw)

def prefill(**over):
    d = prefill_desc(**over)
    return L.kda_linear_prefill(ctypes.byref(d), 8 << 40, 1 << 40, None)

def decode(**over):
    kw = dict(dtype=2, n_seqs=3, n_heads=4, dk=64, dv=128, state=6 << 40, q=1 << 40, k=2 << 40, v=3 << 40,
              g=4 << 40, o=5 << 40)
    kw.update(over)
    d = al.make(al.LinearDecodeDesc, **kw)
    return L.kda_linear_decode(ctypes.byref(d), None)

def gated(**over):
    kw = dict(dtype=2, dim=128, rows=9, x=1 << 40, y=1 << 40)
    kw.update(over)
    d = al.make(al.GatedNormDesc, **kw)
    return L.kda_gated_norm(ctypes.byref(d), None)

def block(**over):
    kw = dict(dtype=2, dim=4096, rows=9, scale=1.0, x=1 << 40, r=2 << 40, r_out=2 << 40)
    kw.update(over)
    d = al.make(al.BlockNormDesc, **kw)
    return L.kda_block_norm(ctypes.byref(d), None)

def kernels():
    return [ln.split()[0] for ln in fake.fake_log().decode().splitlines()]

def reset(older=0, status=0, fails_from=1 << 30):
    fake.fake_reset(older, status, fails_from)

def needs(**over):
    return L.kda_linear_workspace_bytes(ctypes.byref(prefill_desc(**over)), None)

# a prefill that splits sequences needs a workspace, and three launches
CALLS = [(prefill, over, 3 if needs(**over) else 1) for over in (
             dict(), dict(t_total=32768), dict(dtype=1, t_total=5000), dict(n_seqs=24), dict(t_total=64))]
assert sorted(n for _, _, n in CALLS) == [1, 1, 3, 3, 3]
CALLS += [(decode, dict(), 1), (decode, dict(n_seqs=500), 1), (gated, dict(), 1), (gated, dict(dtype=1, dim=1000), 1),
          (block, dict(), 1)]
"""


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("fake_hip")
    fake = str(tmp / "libfake_hip.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", os.path.join(ROOT, "tests", "fake_hip.cpp"),
                    "-o", fake], check=True)

    def run(body):
        script = tmp / "child.py"
        script.write_text(CHILD.format(root=ROOT, fake=fake) + body + "\nprint('child ok')\n")
        preload = " ".join(x for x in (fake, os.environ.get("LD_PRELOAD")) if x)
        p = subprocess.run([sys.executable, str(script)], env=dict(os.environ, LD_PRELOAD=preload),
                           capture_output=True, text=True, timeout=120)
        assert p.returncode == 0 and "child ok" in p.stdout, p.stdout + p.stderr

    return run


def test_an_older_error_is_not_a_launch_s_own(child):
    """An error that an earlier HIP call of the thread left neither fails a good
    launch nor is taken from whoever looks for it."""
    child("""
for call, over, n in CALLS:
    reset(older=101)
    assert call(**over) == 0, (call.__name__, over)
    assert len(kernels()) == n and fake.fake_older() == 101, (call.__name__, over, kernels())
""")


def test_a_launch_that_fails_ends_the_call(child):
    """Its error is the call's, no launch follows it, and none is left behind."""
    child("""
for call, over, n in CALLS:
    for at in range(n):
        reset(status=719, fails_from=at)
        assert call(**over) == -7 and L.kda_last_hip_error() == 719, (call.__name__, over)
        assert len(kernels()) == at + 1 and fake.fake_older() == 0, (call.__name__, over, kernels())
""")


def test_a_segment_past_32_bits_is_refused(child):
    """Segments grow with tokens x heads x dv; where their length leaves 32 bits
    the call is refused (such tensors fit no memory), not divided by zero."""
    child("""
p = [x << 54 for x in range(1, 6)]
big = dict(zip("qkvgo", p), t_total=1 << 30, n_heads=2048, n_k_heads=1, dk=32, h0=None, ht=None, cu_seqlens=None)
for over, want in ((dict(), -2), (dict(n_heads=4096, dv=64), -2), (dict(t_total=1 << 31), -2),
                   (dict(t_total=(1 << 31) - 65, n_heads=65535, n_k_heads=1, dv=32), -2),
                   (dict(n_heads=1024), -2),  # tokens x heads x dv / 32 / 2,048 = 2^31
                   (dict(n_heads=1024, t_total=(1 << 30) - 64), 0), (dict(n_heads=512), 0)):
    kw = dict(big, **over)
    st = ctypes.c_int(9)
    reset()
    L.kda_linear_workspace_bytes(ctypes.byref(prefill_desc(**kw)), ctypes.byref(st))
    assert st.value == want, over
    assert prefill(**kw) == want, over
    assert (len(kernels()) > 0) == (want == 0), over
""")


def test_which_prefill_kernels_the_gpu_tests_reach(child):
    """The sizes of test_gpu_linear_kernels.py enqueue what they are named after,
    and together every instance that a call can reach."""
    child("""
import re
sys.path[:0] = [{tests!r}]
import linear_kernel_cases as lk
seen = set()
for dtype, kind in lk.KINDS:
    for dk, dv, H, Hk in lk.DIMS:
        lengths = lk.lengths_of(dtype, kind, H)
        reset()
        assert prefill(dtype=2 if dtype == "bf16" else 1, n_seqs=len(lengths), t_total=sum(lengths), n_heads=H,
                       n_k_heads=Hk, dk=dk, dv=dv) == 0
        hg = lk.heads_a_workgroup(dv, H, Hk)
        got = [re.findall(r"linear_kernelI(?:DF16b|u6__bf16|f)Li(\\d+)ELi(\\d+)ELi(\\d+)ELi(\\d+)ELb([01])E", k)
               for k in kernels()]
        got = [tuple(int(x) for x in m[0]) for m in got if m]
        chunk = 64 if dtype == "bf16" and kind != "few" else 32
        want = [(chunk, dk, dv * hg, hg, 1)]
        if kind == "split":
            want = [(chunk, dk, dv * hg, hg, 0)] + want
        assert got == want, (dtype, kind, dk, dv, H, Hk, kernels())
        seen |= {{(dtype,) + w for w in want}}
# bf16: outputs in both chunk lengths and the segment pass; fp32: outputs and the segment pass
assert len(seen) == 15 * 3 + 15 * 2, len(seen)
""".format(tests=os.path.join(ROOT, "tests")))
