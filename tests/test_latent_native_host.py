"""What the module _fast_latent hands to the library and does with its answers, without
a GPU: built from its own source for CPU tensors and with stand-ins for the library's
entry points (native_latent_on_host.cpp)."""
import ctypes
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sysconfig

import pytest
import torch

from gated_delta_rule_55_amd import _abi_latent as al
from gated_delta_rule_55_amd.layer import _DTYPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not (shutil.which("g++") and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))),
    reason="needs g++ and Python's headers")

DESC = {"latent_prefill": al.LatentPrefillDesc, "latent_attend": al.LatentAttendDesc, "latent_append": al.LatentAppendDesc, "rotary": al.RotaryDesc}


@pytest.fixture(scope="module")
def fast(tmp_path_factory):
    from gated_delta_rule_55_amd import _abi, build

    if not os.path.exists(_abi.LIB_PATH):
        pytest.skip("libkda.so not built")  # KdaError asks it for its texts
    out = str(tmp_path_factory.mktemp("native") / "_fast_latent.so")
    flags = build._fast_command()
    head = [f for f in flags if f.startswith(("-I", "-isystem", "-D", "-std"))]
    libs = [f for f in flags if f.startswith(("-L", "-l")) and "libkda" not in f]
    subprocess.run(["g++", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", *head, f"-I{build.CSRC}",
                    os.path.join(ROOT, "tests", "native_latent_on_host.cpp"), "-o", out, *libs], check=True)
    loader = importlib.machinery.ExtensionFileLoader("_fast_latent", out)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fast_latent", loader))
    loader.exec_module(m)
    m.host = ctypes.CDLL(out)
    m.host.host_seen.restype = ctypes.c_void_p
    m.host.host_workspace.restype = ctypes.c_size_t
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


CACHE = torch.zeros(6, 4, 320)
TABLE = torch.zeros(3, 2, dtype=torch.int32)
LENS = i32(3, 0, 7)
FREQ = torch.ones(32, dtype=torch.float64)


def attend(q=None, cache=CACHE, table=TABLE, lens=LENS, cu=None, dc=256, scale=0.1, out=None, workspace=None):
    return "latent_attend", (torch.zeros(3, 2, 320) if q is None else q, cache, table, lens, cu, dc, scale, out, workspace)


def append(cache=CACHE, latent=None, pe=None, table=TABLE, lens=LENS, cu=None, weight=torch.ones(256), eps=1e-6,
           freq=FREQ, interleaved=False, magnitude=1.0, rows=None):
    return "latent_append", (cache, torch.zeros(3, 256) if latent is None else latent,
                             torch.zeros(3, 64) if pe is None else pe, table, lens, cu, weight, eps, freq,
                             interleaved, magnitude, rows)


def rotary(x=None, positions=LENS, freq=FREQ, interleaved=True, magnitude=1.0, out=None):
    return "rotary", (torch.zeros(3, 2, 64) if x is None else x, positions, freq, interleaved, magnitude, out)


KV = torch.zeros(5, 2, 192)
CU, CUK = i32(0, 1, 3), i32(0, 4, 5)


def prefill(q=None, k=KV[..., :64], pe=torch.zeros(5, 32), v=KV[..., 64:], cu=CU, cuk=CUK, scale=None, out=None,
            workspace=None):
    return "latent_prefill", (torch.zeros(3, 2, 96) if q is None else q, k, pe, v, cu, cuk, scale, out, workspace)


CALLS = [prefill(), prefill(scale=0.5, out=torch.zeros(3, 2, 128)), attend(), attend(cu=i32(0, 1, 1, 3), out=torch.zeros(3, 2, 256)), append(), append(weight=None, freq=None),
         rotary(), rotary(out=torch.zeros(3, 2, 64))]
IDS = [f"{n}-{i % 2}" for i, (n, _) in enumerate(CALLS)]


def run(fast, call, status=0):
    fast.host.host_reset(status)
    return getattr(fast, call[0])(*call[1])


def seen(fast, call):
    """The descriptor that the library got."""
    assert run(fast, call) is not None and fast.host.host_calls() == 1
    d = DESC[call[0]].from_buffer_copy(ctypes.string_at(fast.host.host_seen(), ctypes.sizeof(DESC[call[0]])))
    assert d.struct_size == ctypes.sizeof(d) and d.dtype == _DTYPES[torch.float32]
    return d


@pytest.mark.parametrize("call", CALLS, ids=IDS)
def test_a_launch_that_failed_is_not_made_again(fast, call):
    from gated_delta_rule_55_amd import KdaError

    for refusal in (-1, -2, -3, -4, -5, -6, -8, -9):
        assert run(fast, call, refusal) is None and fast.host.host_calls() == 1
        assert fast.host.host_calls_with_gil() == 0
    with pytest.raises(KdaError) as e:
        run(fast, call, -7)
    assert fast.host.host_calls() == 1 and e.value.status == -7 and "kda_" + call[0] in str(e.value)


def test_the_wrapper_passes_the_error_on(fast, monkeypatch):
    """latent.py makes no call of its own after it."""
    from gated_delta_rule_55_amd import KdaError, latent

    monkeypatch.setattr(latent, "_fast_latent", fast)
    monkeypatch.setattr(latent._an, "lib", lambda: pytest.fail("called again"))
    for name, a in CALLS:
        fast.host.host_reset(-7)
        with pytest.raises(KdaError):
            if name in ("latent_append", "latent_prefill"):
                getattr(latent, name)(*a)
            elif name == "rotary":
                latent.rotary(*a)
            elif a[4] is None:
                latent.latent_decode(*a[:4], *a[5:])
            else:
                latent.latent_extend(*a)
        assert fast.host.host_calls() == 1


def test_prefill_descriptor(fast):
    wide, out, rows = torch.zeros(3, 3, 96)[:, 1:], torch.zeros(3, 4, 128)[:, :2], torch.zeros(5, 40)
    d = seen(fast, prefill(q=wide, pe=rows[:, 8:], out=out, scale=0.25))
    assert (d.n_seqs, d.n_heads, d.dn, d.dr, d.dv, d.q_total, d.k_total) == (2, 2, 64, 32, 128, 3, 5)
    assert (d.q, d.q_stride, d.o, d.o_stride) == (wide.data_ptr(), 288, out.data_ptr(), 512)
    assert (d.k, d.k_stride, d.k_head_stride) == (KV.data_ptr(), 384, 192)
    assert (d.v, d.v_stride, d.v_head_stride) == (KV.data_ptr() + 256, 384, 192)
    assert (d.k_pe, d.k_pe_stride) == (rows.data_ptr() + 32, 40)
    assert (d.cu_seqlens, d.cu_seqlens_k, d.scale) == (CU.data_ptr(), CUK.data_ptr(), 0.25)
    assert fast.host.host_workspace() == 32
    d = seen(fast, prefill(q=torch.zeros(5, 2, 96), cu=None, cuk=None))
    assert (d.n_seqs, d.cu_seqlens, d.cu_seqlens_k, d.scale) == (1, None, None, 0) and fast.host.host_workspace() == 0
    d = seen(fast, prefill(q=torch.zeros(5, 2, 96), cuk=None))
    assert (d.n_seqs, d.cu_seqlens, d.cu_seqlens_k) == (2, CU.data_ptr(), None)
    assert run(fast, prefill()).shape == (3, 2, 128) and run(fast, prefill(out=out)) is out
    run(fast, prefill(workspace=torch.zeros(7)))
    assert fast.host.host_workspace() == 28


def test_attend_descriptor(fast):
    wide = torch.zeros(3, 5, 320)[:, 1:3]
    out = torch.zeros(3, 4, 256)[:, :2]
    cache = torch.zeros(6, 5, 328)[:, :4, :320]
    d = seen(fast, attend(q=wide, cache=cache, cu=i32(0, 1, 1, 3), out=out))
    assert (d.n_seqs, d.n_heads, d.dc, d.dr, d.page_size, d.max_pages, d.n_pages, d.t_total) == (3, 2, 256, 64, 4, 2, 6, 3)
    assert (d.q, d.q_stride, d.o, d.o_stride) == (wide.data_ptr(), 5 * 320, out.data_ptr(), 4 * 256)
    assert (d.cache, d.page_stride, d.row_stride) == (cache.data_ptr(), 5 * 328, 328)
    assert d.block_table == TABLE.data_ptr() and d.seq_lens == LENS.data_ptr() and d.cu_seqlens
    assert d.scale == ctypes.c_float(0.1).value and fast.host.host_workspace() == 64
    run(fast, attend(workspace=torch.zeros(50, dtype=torch.int32)))
    assert fast.host.host_workspace() == 200
    assert run(fast, attend()).shape == (3, 2, 256)
    assert run(fast, attend(out=out)) is out


def test_append_descriptor(fast):
    rows = torch.zeros(3, 400)
    d = seen(fast, append(latent=rows[:, :256], pe=rows[:, 256:320], rows=rows[:, :320], interleaved=True,
                          magnitude=2.0, eps=1e-5))
    assert (d.latent, d.latent_stride, d.k_pe, d.k_pe_stride) == (rows.data_ptr(), 400, rows.data_ptr() + 1024, 400)
    assert (d.rows_out, d.rows_out_stride) == (rows.data_ptr(), 400)
    assert (d.dc, d.dr, d.page_size, d.max_pages, d.n_pages, d.t_total, d.n_seqs) == (256, 64, 4, 2, 6, 3, 3)
    assert d.rotary == al.KDA_ROTARY_INTERLEAVED and d.magnitude == 2 and d.eps == ctypes.c_float(1e-5).value
    assert d.weight and d.frequencies == FREQ.data_ptr()
    d = seen(fast, append(weight=None, freq=None))
    assert not (d.weight or d.frequencies or d.rows_out or d.cu_seqlens) and d.rotary == al.KDA_ROTARY_HALF
    assert run(fast, append()) is CACHE


def test_rotary_descriptor(fast):
    x = torch.zeros(3, 2, 320)
    d = seen(fast, rotary(x=x[:, :, 256:], out=x[:, :, 64:128]))
    assert (d.x, d.x_stride, d.x_head_stride) == (x.data_ptr() + 1024, 640, 320)
    assert (d.y, d.y_stride, d.y_head_stride) == (x.data_ptr() + 256, 640, 320)
    assert (d.n_heads, d.dim, d.t_total, d.rotary, d.magnitude) == (2, 64, 3, al.KDA_ROTARY_INTERLEAVED, 1)
    x = torch.zeros(1, 2, 64).expand(1, 2, 64)  # one row: its stride says nothing
    assert seen(fast, rotary(x=x, positions=i32(5))).x_stride == 128


NOT_TAKEN = [
    prefill(q=torch.zeros(3, 2, 96).bfloat16()), prefill(q=torch.zeros(3, 2, 192)[..., :96]), prefill(q=torch.zeros(3, 1, 96)),
    prefill(q=torch.zeros(3, 96)), prefill(k=KV[:4, :, :64]), prefill(v=KV[:4, :, 64:]), prefill(v=KV[:, :1, 64:]),
    prefill(pe=torch.zeros(5, 64)), prefill(pe=torch.zeros(4, 32)), prefill(pe=torch.zeros(5, 2, 32)),
    prefill(k=KV[:, :1].expand(5, 2, 192)[..., :64]), prefill(k=KV[..., :128:2]), prefill(cu=None), prefill(cuk=None),
    prefill(cu=CU.long()), prefill(cu=CU[None]), prefill(cu=CU[:0]), prefill(cuk=i32(0, 5)), prefill(cuk=CUK.long()),
    prefill(scale=0.0), prefill(scale=1e-60), prefill(scale="1"), prefill(out=torch.zeros(3, 2, 64)),
    prefill(out=torch.zeros(3, 2, 256)[..., :128]), prefill(workspace=3), prefill(workspace=torch.zeros(4, 4)[:, :2]),
    prefill(k=torch.zeros(5, 2, 8), pe=torch.zeros(5, 88)),   # the library names no workspace
    attend(q=torch.zeros(3, 2, 320, dtype=torch.float16)), attend(q=torch.zeros(3, 2, 640)[..., ::2]),
    attend(q=torch.zeros(3, 2, 640)[..., :320]), attend(q=torch.zeros(320, 3, 2).permute(1, 2, 0)),
    attend(q=torch.zeros(1, 2, 320).expand(3, 2, 320)), attend(q=torch.zeros(4, 2, 320)),
    attend(q=torch.zeros(3, 2, 256)), attend(q=torch.zeros(3, 320)), attend(q=None, cache=CACHE.bfloat16()),
    attend(cache=CACHE[0]), attend(cache=CACHE[..., ::2]), attend(cache=CACHE[:1].expand(6, 4, 320)),
    attend(cache=torch.zeros(6, 1, 320).expand(6, 4, 320)), attend(table=TABLE.long()), attend(table=TABLE[:2]),
    attend(table=TABLE[:, ::2]), attend(lens=LENS.long()), attend(lens=i32(1, 2)), attend(cu=i32(0, 1, 3)),
    attend(cu=i32(0, 1, 1, 3).long()), attend(dc=320), attend(dc=0), attend(dc=256.0), attend(dc=2**70), attend(scale="0.1"),
    attend(scale=None), attend(out=torch.zeros(3, 2, 128)), attend(out=torch.zeros(3, 2, 256, dtype=torch.bfloat16)),
    attend(out=torch.zeros(3, 2, 512)[..., :256]), attend(workspace=torch.zeros(8, 8)[:, :4]), attend(workspace=3),
    append(latent=torch.zeros(3, 250)), append(latent=torch.zeros(4, 256)), append(pe=torch.zeros(4, 64)),
    append(pe=torch.zeros(3, 64, dtype=torch.bfloat16)), append(weight=torch.ones(256).bfloat16()),
    append(weight=torch.ones(320)), append(freq=FREQ.float()), append(freq=FREQ[:16]), append(magnitude=0),
    append(magnitude=1e-60), append(rows=torch.zeros(3, 256)), append(rows=torch.zeros(1, 320).expand(3, 320)),
    append(lens=i32(1, 2)), append(cu=i32(0, 3)), append(cache=CACHE[..., :256]),
    rotary(x=torch.zeros(3, 64)), rotary(x=torch.zeros(3, 1, 64).expand(3, 2, 64)), rotary(positions=LENS.long()),
    rotary(positions=i32(1, 2)), rotary(freq=FREQ.float()), rotary(freq=None), rotary(magnitude=0.0),
    rotary(out=torch.zeros(3, 2, 32)), rotary(out=torch.zeros(1, 2, 64).expand(3, 2, 64)), rotary(x=3),
]


@pytest.mark.parametrize("call", NOT_TAKEN, ids=[f"{i}-{n}" for i, (n, _) in enumerate(NOT_TAKEN)])
def test_a_call_that_it_does_not_take_is_handed_back(fast, call):
    """Before the library is asked, which could read its arguments."""
    assert run(fast, call) is None and fast.host.host_calls() == 0


@pytest.mark.parametrize("call", [prefill(), attend(), append(), rotary()], ids=["prefill", "attend", "append", "rotary"])
def test_numbers_of_arguments(fast, call):
    fast.host.host_reset(0)
    f, a = getattr(fast, call[0]), call[1]
    assert f(*a[:-1]) is None and f(*a, None) is None and f() is None and fast.host.host_calls() == 0


def test_no_rows(fast):
    """Nothing to do is taken too: the library says so."""
    none = torch.zeros(0, dtype=torch.int32)
    assert run(fast, prefill(q=torch.zeros(0, 2, 96))).shape == (0, 2, 128)
    assert run(fast, attend(q=torch.zeros(0, 2, 320), table=TABLE[:0], lens=none)).shape == (0, 2, 256)
    assert run(fast, append(latent=torch.zeros(0, 256), pe=torch.zeros(0, 64), table=TABLE[:0], lens=none)) is CACHE
    assert run(fast, rotary(x=torch.zeros(0, 2, 64), positions=none)).shape == (0, 2, 64)
