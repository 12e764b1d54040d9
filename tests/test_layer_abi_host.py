"""The C ABI of linear attention and the norms on the host: exports, struct
sizes, and refusals before anything is launched.  No GPU: every call here fails
validation, sizes a workspace or has nothing to do."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="fake-pointer checks run without a GPU")


@pytest.fixture(scope="module")
def al():
    from gated_delta_rule_55_amd import _abi, _abi_layer

    if not os.path.exists(_abi.LIB_PATH):
        pytest.skip("libkda.so not built")
    return _abi_layer


def test_exports_and_struct_sizes(al, tmp_path):
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in ("kda_linear.h", "kda_norm.h"))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(kda_[a-z0-9_]+)\s*\(", text, flags=re.M)
    assert sorted(names) == ["kda_block_norm", "kda_gated_norm", "kda_linear_decode",
                             "kda_linear_prefill", "kda_linear_workspace_bytes"]
    for n in names:
        assert hasattr(al.lib(), n)
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include "kda_linear.h"\n#include "kda_norm.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu", sizeof(kda_linear_prefill_desc),'
                   ' sizeof(kda_linear_decode_desc), sizeof(kda_gated_norm_desc),'
                   ' sizeof(kda_block_norm_desc));return 0;}\n')
    exe = str(tmp_path / "sz")
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(c) for c in (
        al.LinearPrefillDesc, al.LinearDecodeDesc, al.GatedNormDesc, al.BlockNormDesc)]


def _prefill(al, over):
    kw = dict(dtype=2, n_seqs=2, n_heads=4, n_k_heads=2, dk=64, dv=128, decay=0, t_total=300,
              q=0x1000000, k=0x2000000, v=0x3000000, g=0x4000000, o=0x5000000, h0=0x6000000,
              ht=0x6000000, cu_seqlens=0x7000000)
    kw.update(over)
    d = al.make(al.LinearPrefillDesc, **{a: b for a, b in kw.items() if a != "struct_size"})
    if "struct_size" in over:
        d.struct_size = over["struct_size"]
    return d


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=0), -3), (dict(dtype=3), -3), (dict(n_seqs=0), -2),
    (dict(n_heads=0), -2), (dict(n_heads=65536), -2), (dict(n_k_heads=3), -2), (dict(n_k_heads=-1), -2),
    (dict(n_k_heads=8), -2), (dict(dk=96), -4), (dict(dv=256), -4), (dict(decay=2), -4),
    (dict(t_total=-1), -2), (dict(t_total=1 << 31), -2), (dict(scale=float("nan")), -2),
    (dict(state_dtype=9), -3), (dict(dtype=1, state_dtype=2), -4),
    (dict(n_seqs=1 << 22), -2),                                     # threads of a launch past 32 bits
    (dict(q_stride=64), -2), (dict(k_stride=132), -2), (dict(v_stride=1 << 29), -2),
    (dict(o_stride=-8), -2),
    (dict(state_indices=0x8000000, n_slots=0), -2),
    (dict(state_indices=0x8000000, n_slots=(1 << 31) - 1, n_heads=65535, n_k_heads=0), -2),
    (dict(cu_seqlens=None), -1), (dict(q=None), -1), (dict(g=None), -1), (dict(o=None), -1),
    (dict(q=0x1000008), -5), (dict(o=0x5000002), -5), (dict(h0=0x6000004, ht=None), -5), (dict(g=0x4000002), -5),
    (dict(cu_seqlens=0x7000001), -5), (dict(state_indices=0x8000002, n_slots=4), -5),
    (dict(o=0x1000000), -9), (dict(o=0x3000000 + 1024), -9), (dict(o=0x6000000), -9),
    (dict(ht=0x6000000 + 4096), -9),                                # partly over h0
    (dict(ht=0x2000000, h0=None), -9), (dict(o=0x4000000), -9),
    (dict(o=0x1000000 + 240, q_stride=1024, o_stride=1024), -9),    # the rows of o start in q's
    (dict(o=0x1000000 - 1008, q_stride=1024, o_stride=1024), -9),   # and end in them
    (dict(o=0x1000000 + 256, q_stride=1024, o_stride=1024), -7),    # side by side: launched, no device
    (dict(o=0x1000000 - 1024, q_stride=1024, o_stride=1024), -7),
])
def test_linear_prefill_refuses(al, over, status):
    d = _prefill(al, over)
    assert al.lib().kda_linear_prefill(ctypes.byref(d), 0x9000000, 1 << 40, None) == status


@no_gpu_only
def test_linear_workspace(al):
    import gated_delta_rule_55_amd as kda

    L = al.lib()
    # a call that cannot split a sequence needs none
    assert kda.linear_workspace_bytes(64, 32, 128, 128) == 0
    need = kda.linear_workspace_bytes(32768, 32, 128, 128)
    assert 0 < need < 300 << 20
    d = _prefill(al, dict(t_total=20000, n_heads=2, n_k_heads=0, o=0x15000000, v=0x13000000))
    need = L.kda_linear_workspace_bytes(ctypes.byref(d), None)
    assert need > 0
    assert L.kda_linear_prefill(ctypes.byref(d), None, 0, None) == -6
    assert L.kda_linear_prefill(ctypes.byref(d), 0x90000000, need - 1, None) == -6
    assert L.kda_linear_prefill(ctypes.byref(d), 0x90000010, need, None) == -5
    assert L.kda_linear_prefill(ctypes.byref(d), 0x13000000, need, None) == -9   # over v
    st = ctypes.c_int(0)
    bad = _prefill(al, dict(dk=48))
    assert L.kda_linear_workspace_bytes(ctypes.byref(bad), ctypes.byref(st)) == 0 and st.value == -4
    assert L.kda_linear_prefill(None, None, 0, None) == -1


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=5), -3), (dict(n_seqs=-1), -2), (dict(n_heads=0), -2),
    (dict(n_k_heads=3), -2), (dict(dk=16), -4), (dict(dv=0), -4), (dict(decay=-1), -4),
    (dict(scale=float("inf")), -2), (dict(state_dtype=4), -3), (dict(dtype=1, state_dtype=2), -4),
    (dict(n_seqs=1 << 22), -2), (dict(q_stride=100), -2), (dict(state_indices=0x8000000, n_slots=-1), -2),
    (dict(state=None), -1), (dict(v=None), -1), (dict(g=None), -1), (dict(k=0x2000008), -5),
    (dict(state=0x6000008), -5), (dict(g=0x4000001), -5), (dict(o=0x6000000), -9),
    (dict(o=0x3000000), -9), (dict(state=0x2000000), -9), (dict(n_seqs=0, state=None, q=None), 0),
])
def test_linear_decode_refuses(al, over, status):
    kw = dict(dtype=2, n_seqs=3, n_heads=4, n_k_heads=2, dk=64, dv=128, decay=0, state=0x6000000,
              q=0x1000000, k=0x2000000, v=0x3000000, g=0x4000000, o=0x5000000)
    kw.update(over)
    d = al.make(al.LinearDecodeDesc, **{a: b for a, b in kw.items() if a != "struct_size"})
    if "struct_size" in over:
        d.struct_size = over["struct_size"]
    assert al.lib().kda_linear_decode(ctypes.byref(d), None) == status


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=0), -3), (dict(dim=0), -2), (dict(dim=16385), -2),
    (dict(rows=-1), -2), (dict(rows=1 << 31), -2), (dict(gate=3), -4), (dict(gate_first=2), -4),
    (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(x_stride=99), -2),
    (dict(y_stride=(1 << 28) + 1), -2), (dict(x=None), -1), (dict(y=None), -1), (dict(x=0x1000001), -5),
    (dict(weight=0x2000002), -5), (dict(y=0x1000002), -9), (dict(y=0x1000000, y_stride=200), -9),
    (dict(y=0x3000000 + 200), -9), (dict(y=0x2000000), -9),
    (dict(y=0x1000000 + 198, x_stride=256, y_stride=256), -9),
    (dict(y=0x1000000 + 200, x_stride=256, y_stride=256), -7), (dict(rows=0, x=None, y=None), 0),
])
def test_gated_norm_refuses(al, over, status):
    kw = dict(dtype=2, dim=100, gate=2, rows=7, eps=1e-6, x=0x1000000, weight=0x2000000, z=0x3000000,
              y=0x4000000)
    kw.update(over)
    d = al.make(al.GatedNormDesc, **{a: b for a, b in kw.items() if a != "struct_size"})
    if "struct_size" in over:
        d.struct_size = over["struct_size"]
    assert al.lib().kda_gated_norm(ctypes.byref(d), None) == status


@no_gpu_only
@pytest.mark.parametrize("over,status", [
    (dict(struct_size=8), -8), (dict(dtype=0), -3), (dict(residual_dtype=7), -3),
    (dict(dtype=1, residual_dtype=2), -4), (dict(dim=0), -2), (dict(dim=16385), -2), (dict(rows=-1), -2),
    (dict(gate=-1), -4), (dict(eps=-1e-9), -2), (dict(scale=float("inf")), -2), (dict(r_stride=5), -2),
    (dict(x=None), -1), (dict(r=None), -1), (dict(r_out=None), -1), (dict(y=None), -1),
    (dict(w_pre=None), -1), (dict(r=0x2000002, residual_dtype=1), -5), (dict(c=0x5000001), -5),
    (dict(r_out=0x1000000), -9), (dict(r_out=0x2000002), -9), (dict(r_out=0x2000000, r_out_stride=128), -9),
    (dict(y=0x2000000), -9), (dict(y=0x7000000), -9), (dict(y=0x1000000, y_stride=104), -9),
    (dict(y=0x3000000), -9), (dict(r_out=0x6000000), -9), (dict(rows=0, x=None), 0),
])
def test_block_norm_refuses(al, over, status):
    kw = dict(dtype=2, dim=100, gate=1, rows=9, eps=1e-6, scale=1.0, x=0x1000000, r=0x2000000,
              w_post=0x3000000, w_pre=0x4000000, c=0x5000000, z=0x6000000, r_out=0x7000000, y=0x8000000)
    kw.update(over)
    d = al.make(al.BlockNormDesc, **{a: b for a, b in kw.items() if a != "struct_size"})
    if "struct_size" in over:
        d.struct_size = over["struct_size"]
    assert al.lib().kda_block_norm(ctypes.byref(d), None) == status


def test_wrappers_refuse_cpu_tensors():
    import gated_delta_rule_55_amd as kda

    x = torch.zeros(4, 2, 32)
    with pytest.raises(ValueError, match="GPU only"):
        kda.linear_prefill(x, x, x, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU only"):
        kda.linear_decode(torch.zeros(4, 2, 32, 32), x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="GPU only"):
        kda.gated_norm(x)
    with pytest.raises(ValueError, match="GPU only"):
        kda.block_norm(x, x)
    with pytest.raises(TypeError):
        kda.gated_norm(None)


def test_row_strides_of_views():
    """The row check on the CPU: which views have their rows at one stride."""
    from gated_delta_rule_55_amd import layer

    big = torch.zeros(6, 4, 40)
    dev = big.device

    def stride(t):
        return layer._rows(t, "t", t.shape, torch.float32, dev)[1]

    assert stride(big) == 0
    assert stride(big[:, :, :16]) == 40                      # heads at one stride
    assert stride(big[:, 1, :]) == 160
    assert stride(big[::2, 1:2, :8]) == 320
    for bad in (big[:, :2], big[:, ::2], big.transpose(0, 1), big.transpose(1, 2), big[:, :1].expand(6, 4, 40)):
        if bad.is_contiguous():
            continue
        ok = bad.shape[1] == 2 and bad.stride(1) * 2 == bad.stride(0)
        if ok:
            assert stride(bad) == bad.stride(1)
        else:
            with pytest.raises(ValueError):
                stride(bad)
    q = torch.zeros(5, 96)
    assert layer._rows3(q[:, 32:64].view(5, 1, 32), "q", (5, 1, 32), torch.float32, dev)[1] == 96
    with pytest.raises(ValueError):
        layer._rows3(torch.zeros(5, 32, 2).transpose(1, 2), "q", (5, 2, 32), torch.float32, dev)
    with pytest.raises(ValueError):
        layer._rows3(torch.zeros(1, 1, 32).expand(5, 2, 32), "q", (5, 2, 32), torch.float32, dev)


def test_packed_descriptors_match_the_structures(al):
    """struct.pack and the ctypes structures lay out the same bytes."""
    vals = dict(al.LinearDecodeDesc._fields_)
    for fmt, cls in ((al.LINEAR_DECODE, al.LinearDecodeDesc), (al.GATED_NORM, al.GatedNormDesc),
                     (al.BLOCK_NORM, al.BlockNormDesc)):
        args = [i + 0.5 if t is ctypes.c_float else i + 3 for i, (_, t) in enumerate(cls._fields_)]
        assert fmt.pack(*args) == bytes(cls(*args))
    assert vals["n_slots"] is ctypes.c_int32
