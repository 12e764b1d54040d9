"""The C ABI of latent attention on the host: exports, struct sizes, and refusals before
anything is launched.  No GPU: every call here fails validation, sizes a workspace or has
nothing to do, or ends at the launch without a device (-7)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="fake-pointer checks run without a GPU")
NAN, INF = float("nan"), float("inf")
I32 = (1 << 31) - 1


@pytest.fixture(scope="module")
def al():
    from gated_delta_rule_55_amd import _abi, _abi_latent

    if not os.path.exists(_abi.LIB_PATH):
        pytest.skip("libkda.so not built")
    return _abi_latent


def test_exports_and_struct_sizes(al, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda_latent.h")).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(kda_[a-z0-9_]+)\s*\(", text, flags=re.M)
    assert sorted(names) == ["kda_latent_append", "kda_latent_attend", "kda_latent_prefill",
                             "kda_latent_prefill_workspace_bytes", "kda_latent_workspace_bytes", "kda_rotary"]
    for n in names:
        assert hasattr(al.lib(), n)
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include "kda_latent.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu", sizeof(kda_latent_prefill_desc),'
                   ' sizeof(kda_latent_attend_desc), sizeof(kda_latent_append_desc),'
                   ' sizeof(kda_rotary_desc));return 0;}\n')
    exe = str(tmp_path / "sz")
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(c) for c in (
        al.LatentPrefillDesc, al.LatentAttendDesc, al.LatentAppendDesc, al.RotaryDesc)]


def desc(al, cls, base, over):
    kw = dict(base, **over)
    d = al.make(cls, **{a: b for a, b in kw.items() if a != "struct_size"})
    if "struct_size" in over:
        d.struct_size = over["struct_size"]
    return d


# a workspace of a prefill of these sizes: 300 queries, 700 keys, 4 heads
PREFILL = dict(dtype=2, n_seqs=2, n_heads=4, dn=128, dr=64, dv=128, q_total=300, k_total=700, q=0x1000000, k=0x2000000,
               k_pe=0x3000000, v=0x4000000, o=0x5000000, cu_seqlens=0x6000000, cu_seqlens_k=0x6001000)


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=0), -3), (dict(dtype=3), -3), (dict(n_seqs=0), -2), (dict(n_heads=0), -2),
    (dict(n_heads=65536), -2), (dict(q_total=-1), -2), (dict(k_total=-1), -2), (dict(q_total=I32 - 63), -2),
    (dict(k_total=I32 - 63), -2), (dict(q_total=1 << 30, n_heads=16), -2), (dict(n_seqs=1 << 23), -2),
    (dict(dn=96), -4), (dict(dv=32), -4), (dict(dr=128), -4), (dict(dr=0), -4),
    (dict(scale=-1.0), -2), (dict(scale=NAN), -2), (dict(scale=INF), -2), (dict(scale=1e-40), -2), (dict(scale=3e38), -2),
    (dict(cu_seqlens_k=None), -2),   # other keys than queries
    (dict(q_stride=760), -2), (dict(q_stride=772), -2), (dict(k_stride=500), -2), (dict(k_head_stride=120), -2),
    (dict(k_head_stride=132), -2), (dict(v_stride=-8), -2), (dict(k_stride=(1 << 22) + 8), -2),
    (dict(o_stride=(1 << 22) + 8), -2), (dict(k_pe_stride=(1 << 22) + 8), -2), (dict(q_stride=(1 << 28) + 8), -2),
    (dict(n_heads=65535, q_total=300, dn=128), -2),   # dense rows of k past 2^22
    (dict(cu_seqlens=None), -1), (dict(cu_seqlens=None, cu_seqlens_k=None, k_total=300), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(k_pe=None), -1), (dict(v=None), -1), (dict(o=None), -1),
    (dict(q=0x1000008), -5), (dict(k=0x2000004), -5), (dict(k_pe=0x3000002), -5), (dict(v=0x4000008), -5),
    (dict(o=0x5000008), -5), (dict(cu_seqlens=0x6000002), -5), (dict(cu_seqlens_k=0x6001001), -5),
    (dict(o=0x1000000), -9), (dict(o=0x2000000 + 16), -9), (dict(o=0x3000000), -9), (dict(o=0x4000000 + 1024), -9),
    (dict(o=0x6000000 - 16), -9), (dict(cu_seqlens_k=0x5000000), -9),
    (dict(o=0x1000000 + 1536, q_stride=2048, o_stride=2048), -7),      # beside q in one row: launched, no device
    (dict(o=0x1000000 + 1520, q_stride=2048, o_stride=2048), -9),
    (dict(k_head_stride=256, v_head_stride=256, v=0x2000000 + 256), -7), (dict(q_total=0, q=None, o=None), 0),
])
def test_prefill_refuses(al, over, status):
    d = desc(al, al.LatentPrefillDesc, PREFILL, over)
    assert al.lib().kda_latent_prefill(ctypes.byref(d), 0x90000000, 1 << 40, None) == status


@no_gpu_only
def test_prefill_workspace(al):
    import gated_delta_rule_55_amd as kda

    L = al.lib()
    d = desc(al, al.LatentPrefillDesc, PREFILL, {})
    st = ctypes.c_int(5)
    need = L.kda_latent_prefill_workspace_bytes(ctypes.byref(d), ctypes.byref(st))
    # whole parts of [300 queries, 4 heads] of 128 sums, a maximum and a sum
    assert st.value == 0 and need > 0 and need % (300 * 4 * (128 * 4 + 8)) == 0
    assert need == kda.latent_prefill_workspace_bytes(300, 700, 4, 128, 64, 128, 2)
    f = L.kda_latent_prefill
    assert f(ctypes.byref(d), None, 0, None) == -6 and f(ctypes.byref(d), 0x90000000, need - 1, None) == -6
    assert f(ctypes.byref(d), 0x90000010, need, None) == -5
    for at in (0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000):   # over q, k, k_pe, v, o, cu
        assert f(ctypes.byref(d), at, need, None) == -9
    assert f(ctypes.byref(d), 0x90000000, need, None) == -7
    # a call that fills the GPU, and one without queries, need none
    for over in (dict(q_total=40000, k_total=40000, n_heads=32, q_stride=0), dict(q_total=0)):
        d = desc(al, al.LatentPrefillDesc, PREFILL, over)
        assert L.kda_latent_prefill_workspace_bytes(ctypes.byref(d), None) == 0
    bad = desc(al, al.LatentPrefillDesc, PREFILL, dict(dn=48))
    assert L.kda_latent_prefill_workspace_bytes(ctypes.byref(bad), ctypes.byref(st)) == 0 and st.value == -4
    assert f(None, None, 0, None) == -1
    # never above a share for every workgroup that runs at a time
    for T in (1, 127, 128, 1000, 30000):
        for H in (1, 7, 128):
            for dt in (torch.float32, torch.bfloat16):
                n = kda.latent_prefill_workspace_bytes(T, 1 << 20, H, 128, 64, 128, 1, dt)
                assert n <= 512 * 128 * (128 * 4 + 8)


ATTEND = dict(dtype=2, n_seqs=3, n_heads=4, dc=512, dr=64, page_size=64, max_pages=8, n_pages=20, scale=0.1, t_total=9,
              q=0x1000000, cache=0x2000000, o=0x5000000, block_table=0x6000000, seq_lens=0x6001000,
              cu_seqlens=0x6002000)


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=5), -3), (dict(n_seqs=-1), -2), (dict(n_seqs=(1 << 24) + 1), -2),
    (dict(n_heads=0), -2), (dict(n_heads=65536), -2), (dict(dc=128), -4), (dict(dc=0), -4), (dict(dr=16), -4),
    (dict(page_size=0), -2), (dict(max_pages=0), -2), (dict(n_pages=-1), -2), (dict(page_size=I32, max_pages=2), -2),
    (dict(page_size=I32 - 255, max_pages=1), -2), (dict(t_total=-1), -2), (dict(t_total=I32 // 4), -2),
    (dict(scale=0.0), -2), (dict(scale=-0.1), -2), (dict(scale=NAN), -2), (dict(scale=INF), -2), (dict(scale=1e-39), -2),
    (dict(scale=3e38), -2),
    (dict(cu_seqlens=None), -2),     # 9 tokens of 3 sequences
    (dict(q_stride=2296), -2), (dict(q_stride=2308), -2), (dict(o_stride=2040), -2), (dict(o_stride=(1 << 22) + 8), -2),
    (dict(row_stride=568), -2), (dict(row_stride=580), -2), (dict(page_stride=64 * 576 - 8), -2),
    (dict(page_stride=64 * 576 + 4), -2), (dict(page_stride=1 << 41), -2),
    (dict(q=None), -1), (dict(o=None), -1), (dict(cache=None), -1), (dict(block_table=None), -1), (dict(seq_lens=None), -1),
    (dict(q=0x1000008), -5), (dict(cache=0x2000002), -5), (dict(o=0x5000004), -5), (dict(block_table=0x6000002), -5),
    (dict(seq_lens=0x6001001), -5), (dict(cu_seqlens=0x6002002), -5),
    (dict(o=0x1000000), -9), (dict(o=0x2000000 + 4096), -9), (dict(o=0x6000000), -9), (dict(o=0x6001000 - 16), -9),
    (dict(o=0x6002000), -9), (dict(o=0x1000000 + 2304 * 2, q_stride=8192, o_stride=8192), -7),
    (dict(n_pages=0, cache=None), -7), (dict(n_seqs=0, t_total=0, q=None, o=None), 0), (dict(t_total=0, q=None), 0),
    (dict(cu_seqlens=None, t_total=3), -7),
])
def test_attend_refuses(al, over, status):
    d = desc(al, al.LatentAttendDesc, ATTEND, over)
    assert al.lib().kda_latent_attend(ctypes.byref(d), 0x90000000, 1 << 40, None) == status


@no_gpu_only
def test_attend_workspace(al):
    import gated_delta_rule_55_amd as kda

    L = al.lib()
    d = desc(al, al.LatentAttendDesc, ATTEND, {})
    need = L.kda_latent_workspace_bytes(ctypes.byref(d), None)
    assert need == kda.latent_workspace_bytes(9, 4, 512, 64, 3, 8, 64, extend=True) > 0
    f = L.kda_latent_attend
    assert f(ctypes.byref(d), None, 0, None) == -6 and f(ctypes.byref(d), 0x90000000, need - 1, None) == -6
    assert f(ctypes.byref(d), 0x90000080, need, None) == -5
    for at in (0x1000000, 0x2000000, 0x5000000, 0x6000000, 0x6001000, 0x6002000 - 256):
        assert f(ctypes.byref(d), at, need, None) == -9
    st = ctypes.c_int(0)
    bad = desc(al, al.LatentAttendDesc, ATTEND, dict(dc=100))
    assert L.kda_latent_workspace_bytes(ctypes.byref(bad), ctypes.byref(st)) == 0 and st.value == -4
    assert f(None, None, 0, None) == -1 and L.kda_latent_workspace_bytes(None, ctypes.byref(st)) == 0 and st.value == -1
    # sums of two pieces a workgroup: the same for long caches as for short ones
    long = kda.latent_workspace_bytes(64, 128, 512, 64, 64, 10000, 64)
    assert long < 300 << 20 and kda.latent_workspace_bytes(64, 128, 512, 64, 64, 1000, 64) == long


APPEND = dict(dtype=2, n_seqs=3, dc=512, dr=64, page_size=64, max_pages=8, n_pages=20, rotary=0, eps=1e-6, t_total=9,
              latent=0x1000000, k_pe=0x1100000, cache=0x2000000, rows_out=0x3000000, weight=0x4000000,
              frequencies=0x4100000, block_table=0x6000000, seq_lens=0x6001000, cu_seqlens=0x6002000)


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=0), -3), (dict(n_seqs=-1), -2), (dict(dc=1024), -4), (dict(dr=96), -4),
    (dict(page_size=0), -2), (dict(max_pages=-1), -2), (dict(n_pages=-1), -2), (dict(t_total=-1), -2),
    (dict(t_total=1 << 25), -2),     # threads of a launch past 2^31
    (dict(rotary=2), -4), (dict(rotary=-1), -4), (dict(eps=-1.0), -2), (dict(eps=NAN), -2), (dict(eps=INF), -2),
    (dict(magnitude=NAN), -2), (dict(magnitude=INF), -2), (dict(cu_seqlens=None), -2),
    (dict(latent_stride=504), -2), (dict(k_pe_stride=68), -2), (dict(rows_out_stride=568), -2), (dict(row_stride=512), -2),
    (dict(latent=None), -1), (dict(k_pe=None), -1), (dict(cache=None), -1), (dict(block_table=None), -1),
    (dict(seq_lens=None), -1), (dict(latent=0x1000008), -5), (dict(k_pe=0x1100002), -5), (dict(rows_out=0x3000004), -5),
    (dict(cache=0x2000008), -5), (dict(weight=0x4000002), -5), (dict(frequencies=0x4100004), -5),
    (dict(block_table=0x6000001), -5), (dict(cache=0x1000000), -9), (dict(cache=0x1100000 - 64), -9),
    (dict(cache=0x3000000), -9), (dict(cache=0x4000000), -9), (dict(cache=0x6002000 - 16), -9),
    (dict(rows_out=0x1000000), -9), (dict(rows_out=0x1100000), -9), (dict(rows_out=0x4000000), -9),
    (dict(rows_out=0x4100000), -9), (dict(rows_out=0x6001000), -9),
    (dict(k_pe=0x1000000 + 1024, latent_stride=576, k_pe_stride=576, rows_out=0x1000000), -7),      # in place
    (dict(k_pe=0x1000000 + 1024, latent_stride=576, k_pe_stride=576, rows_out=0x1000010), -9),
    (dict(k_pe=0x1000000 + 1024, latent_stride=640, k_pe_stride=640, rows_out=0x1000000), -9),      # other strides
    (dict(rows_out=None, weight=None, frequencies=None), -7), (dict(n_pages=0, cache=None), -7),
    (dict(t_total=0, latent=None), 0), (dict(n_seqs=0, t_total=0, latent=None, cache=None), 0),
])
def test_append_refuses(al, over, status):
    d = desc(al, al.LatentAppendDesc, APPEND, over)
    assert al.lib().kda_latent_append(ctypes.byref(d), None) == status
    assert al.lib().kda_latent_append(None, None) == -1


ROTARY = dict(dtype=2, n_heads=4, dim=64, rotary=1, t_total=9, x=0x1000000, y=0x2000000, positions=0x3000000,
              frequencies=0x3001000)


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=7), -3), (dict(n_heads=0), -2), (dict(n_heads=65536), -2), (dict(dim=0), -4),
    (dict(dim=24), -4), (dict(dim=272), -4), (dict(dim=8), -4), (dict(rotary=3), -4), (dict(t_total=-1), -2),
    (dict(t_total=I32), -2), (dict(t_total=I32 - 64, n_heads=8, dim=256), -2), (dict(magnitude=NAN), -2),
    (dict(magnitude=-INF), -2), (dict(x_stride=248), -2), (dict(x_head_stride=56), -2), (dict(y_head_stride=68), -2),
    (dict(y_stride=260), -2), (dict(x_head_stride=128, x_stride=440), -2), (dict(x_stride=(1 << 28) + 8), -2),
    (dict(x=None), -1), (dict(y=None), -1), (dict(positions=None), -1), (dict(frequencies=None), -1),
    (dict(x=0x1000008), -5), (dict(y=0x2000002), -5), (dict(positions=0x3000002), -5), (dict(frequencies=0x3001004), -5),
    (dict(y=0x1000000), -7), (dict(y=0x1000010), -9), (dict(y=0x1000000, y_stride=320), -9),
    (dict(y=0x1000000 + 128, x_head_stride=128, y_head_stride=128), -7),     # the other half of each head
    (dict(y=0x1000000 + 112, x_head_stride=128, y_head_stride=128), -9), (dict(y=0x3000000), -9), (dict(y=0x3001000), -9),
    (dict(t_total=0, x=None), 0),
])
def test_rotary_refuses(al, over, status):
    d = desc(al, al.RotaryDesc, ROTARY, over)
    assert al.lib().kda_rotary(ctypes.byref(d), None) == status
    assert al.lib().kda_rotary(None, None) == -1


def test_python_refuses_what_the_abi_cannot_see():
    """CPU tensors, other types and shapes: refused by name before the library is called."""
    import gated_delta_rule_55_amd as kda

    x, i = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.rotary(x, i, torch.zeros(32, dtype=torch.float64)),
                 lambda: kda.latent_prefill(x, x, x[:, 0], x),
                 lambda: kda.latent_decode(x, x, i[None], i, 32, 1.0),
                 lambda: kda.latent_append(x, x[:, 0], x[:, 0], i[None], i)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
    with pytest.raises(TypeError):
        kda.rotary(3, i, i)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.latent_extend(x, x, i[None], i, None, 32, 1.0)
    for bad in (0.0, -1.0, NAN, INF, 1e-40):
        with pytest.raises(ValueError, match="scale"):
            kda.latent._positive(bad)
    for bad in (0.0, NAN, INF, 1e-60):
        with pytest.raises(ValueError, match="magnitude"):
            kda.latent._magnitude(bad)
    with pytest.raises(kda.KdaError):
        kda.latent_workspace_bytes(1, 1, 100, 64, 1, 1, 64)


def test_rotary_frequencies():
    import gated_delta_rule_55_amd as kda

    f = kda.rotary_frequencies(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(kda.rotary_frequencies(64, factor=4.0), f / 4)
    g = kda.rotary_frequencies(64, factor=40.0, original_length=4096)
    turns = 4096 * f / (2 * torch.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 40, rtol=1e-15)
    middle = (turns > 1) & (turns < 32)
    keep = (turns[middle] - 1) / 31
    assert middle.any() and torch.allclose(g[middle], f[middle] * (keep + (1 - keep) / 40), rtol=1e-14)
    for bad in (dict(dim=0), dict(dim=7), dict(dim=64, base=0), dict(dim=64, factor=-1.0), dict(dim=64, slow=2, fast=1),
                dict(dim=64, original_length=0)):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(**bad)
