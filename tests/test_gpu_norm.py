"""The gated norm and the block norm on the GPU against the fp64 oracle.

Bounds (u: half a step of a type, layer_cases.py).  The kernels sum dim squares
in fp32 (at most dim u_fp32 relative, all terms positive, halved by the root)
and do at most 12 further fp32 operations and one exponential a value, whose
argument's rounding adds |z| steps: s = (dim / 2 + 20 + 2 |z|) u_fp32 relative
on a product of factors.  Then the result is rounded once.
A sum r' = r + p carries p's error, and one more step of each term.  y, its
norm, carries r''s error: elementwise through the numerator, and through the
mean square at most by the largest relative change of the row's norm."""
import numpy as np
import pytest
import torch

import oracle
from layer_cases import F32 as U32
from layer_cases import U, host64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DIMS = [1, 7, 8, 32, 63, 64, 100, 128, 250, 256, 512, 513, 1000, 1024, 2048, 2050, 4096, 4097, 8192, 16384]


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def draw(seed, *shape, dtype=F32, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=gen)).to(dtype)


def c(t):
    return None if t is None else t.cuda()


def h(t):
    return None if t is None else host64(t)


def check_gated(x, w, z, act, first, eps, y):
    ref = oracle.gated_norm(h(x), h(w), h(z), act, first, eps)
    s = (x.shape[-1] / 2 + 20 + (0 if z is None else 2 * np.abs(h(z)))) * U32
    if first and z is not None:
        s = np.max(s, axis=-1, keepdims=True) * 2  # every gate's error reaches the mean square
    bound = (s + 1.01 * U[x.dtype]) * np.abs(ref) + 1e-37
    off = np.abs(host64(y) - ref)
    assert np.all(off <= bound), np.max(off / bound)


def check_block(x, r, wpost, wpre, z, act, cs, scale, eps, ro, y):
    rr, yy = oracle.block_norm(h(x), h(r), h(wpost), h(wpre), h(z), act, h(cs), scale, eps)
    p = rr - h(r)
    s = (x.shape[-1] / 2 + 20 + (0 if z is None else 2 * np.abs(h(z)))) * U32
    er = s * np.abs(p) + U32 * (np.abs(rr) + np.abs(h(r)))  # r' before its rounding
    bound = er + 1.01 * U[r.dtype] * np.abs(rr) + 1e-37
    off = np.abs(host64(ro) - rr)
    assert np.all(off <= bound), np.max(off / bound)
    if wpre is None:
        assert y is None
        return
    ms = np.sqrt(np.mean(rr * rr, -1, keepdims=True) + eps)
    drms = np.sqrt(np.mean(er * er, -1, keepdims=True)) / ms   # relative change of the root mean square
    bound = (1.01 * U[x.dtype] + (x.shape[-1] / 2 + 20) * U32 + 1.01 * drms) * np.abs(yy) \
        + 1.01 * er / ms * np.abs(h(wpre)) + 1e-37
    off = np.abs(host64(y) - yy)
    assert np.all(off <= bound), np.max(off / bound)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", DIMS)
def test_gated_dims(kda, dtype, dim):
    rows = 37 if dim < 4096 else 5
    x, z, w = draw(1, rows, dim, dtype=dtype), draw(2, rows, dim, dtype=dtype), 1 + 0.3 * draw(3, dim)
    check_gated(x, w, z, "sigmoid", False, 1e-6, kda.gated_norm(c(x), c(w), c(z), "sigmoid"))
    check_gated(x, None, z, "silu", True, 1e-5, kda.gated_norm(c(x), None, c(z), "silu", True, 1e-5))
    check_gated(x, w, None, None, False, 1e-6, kda.gated_norm(c(x), c(w)))


@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 16, 17, 5000])
def test_gated_forms_and_rows(kda, act, first, rows):
    x, z, w = draw(4, rows, 3, 64, dtype=BF), draw(5, rows, 3, 64, dtype=BF, scale=4.0), draw(6, 64)
    check_gated(x, w, z, act, first, 1e-6, kda.gated_norm(c(x), c(w), c(z), act, first))


def test_gated_strides_in_place_and_extremes(kda):
    big = draw(7, 50, 3, 144, dtype=BF)
    g = c(big)
    x, z = g[:, :, :64], g[:, :, 64:128]
    want = (big[:, :, :64], None, big[:, :, 64:128], "sigmoid", False, 1e-6)
    y = kda.gated_norm(x, None, z, "sigmoid")
    check_gated(*want, y)
    kda.gated_norm(x, None, z, "sigmoid", out=x)                       # over x
    assert torch.equal(x, y) and torch.equal(g[:, :, 64:].cpu(), big[:, :, 64:])
    # odd offsets and strides: rows at 2-byte alignment
    odd = c(draw(8, 40, 131, dtype=BF))
    out = torch.zeros(40, 133, dtype=BF, device="cuda")
    kda.gated_norm(odd[:, 1:130], out=out[:, 3:132])
    check_gated(odd[:, 1:130].cpu(), None, None, None, False, 1e-6, out[:, 3:132])
    assert torch.all(out[:, :3] == 0) and torch.all(out[:, 132:] == 0)
    # zero rows, gates at both ends, rows with values that are not finite
    x, z = torch.zeros(6, 32), torch.zeros(6, 32)
    x[1:], z[2], z[3] = draw(9, 5, 32), -200.0, 200.0
    x[4, 5], x[5, 2] = float("inf"), float("nan")
    y = kda.gated_norm(c(x), None, c(z), "sigmoid").cpu()
    assert torch.all(y[0] == 0) and torch.all(y[2] == 0)
    check_gated(x[1:4:2], None, z[1:4:2], "sigmoid", False, 1e-6, y[1:4:2])
    assert torch.isnan(y[4, 5]) and torch.all(y[4, :5] == 0) and torch.all(torch.isnan(y[5]))
    assert kda.gated_norm(torch.zeros(0, 8, device="cuda")).shape == (0, 8)


@pytest.mark.parametrize("dtype,rd", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("dim", DIMS)
def test_block_dims(kda, dtype, rd, dim):
    rows = 33 if dim < 4096 else 5
    x, z, r = draw(10, rows, dim, dtype=dtype), draw(11, rows, dim, dtype=dtype), draw(12, rows, dim, dtype=rd, scale=2.0)
    wpost, wpre, cs = 1 + 0.2 * draw(13, dim), 1 + 0.2 * draw(14, dim), draw(15, dim)
    ro, y = kda.block_norm(c(x), c(r), c(wpost), c(wpre), c(z), "sigmoid", c(cs), 0.7)
    check_block(x, r, wpost, wpre, z, "sigmoid", cs, 0.7, 1e-6, ro, y)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", ["off", None, "silu"])
@pytest.mark.parametrize("chan", [False, True])
def test_block_forms(kda, post, pre, gate, chan):
    x, r = draw(16, 130, 96, dtype=BF), draw(17, 130, 96, dtype=F32)
    wpost, wpre, cs = (draw(18, 96) if post else None), (draw(19, 96) if pre else None), (draw(20, 96) if chan else None)
    z = None if gate == "off" else draw(21, 130, 96, dtype=BF)
    act = None if gate == "off" else gate
    ro, y = kda.block_norm(c(x), c(r), c(wpost), c(wpre), c(z), act, c(cs), -1.5, 1e-5)
    check_block(x, r, wpost, wpre, z, act, cs, -1.5, 1e-5, ro, y)


def test_block_in_place_and_many_rows(kda):
    rows, dim = 20000, 264
    x, r, w = draw(22, rows, dim, dtype=BF), draw(23, rows, dim, dtype=BF), draw(24, dim)
    ro, y = kda.block_norm(c(x), c(r), c(w), c(w))
    check_block(x, r, w, w, None, None, None, 1.0, 1e-6, ro, y)
    xd, rd = c(x), c(r)
    r2, y2 = kda.block_norm(xd, rd, c(w), c(w), residual_out=rd, out=xd)
    assert r2 is rd and y2 is xd and torch.equal(r2, ro) and torch.equal(y2, y)
    e = torch.zeros(0, 16, device="cuda")
    assert kda.block_norm(e, e, weight_pre=torch.ones(16, device="cuda"))[1].shape == (0, 16)


def test_refusals(kda):
    x, r = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (dict(residual=r.double()), dict(residual=r[:2]), dict(weight_pre=w.bfloat16()),
                dict(weight_post=w[:32]), dict(gate=x.float()), dict(activation="gelu"), dict(out=x.clone()),
                dict(channel_scale=w.cpu()), dict(x=x.half()), dict(x=x.t().contiguous().t())):
        kw = dict(dict(x=x, residual=r), **bad)
        with pytest.raises((TypeError, ValueError)):
            kda.block_norm(**kw)
    with pytest.raises(kda.KdaError):
        kda.block_norm(x, x.clone(), weight_pre=w, residual_out=x)     # r' over x
    with pytest.raises(kda.KdaError):
        kda.block_norm(x.float(), x)                                   # bf16 residual of fp32 x
    big = torch.zeros(4, 200, dtype=BF, device="cuda")
    with pytest.raises(kda.KdaError):
        kda.gated_norm(big[:, :64], out=big[:, 8:72])                  # partly over x
    with pytest.raises(kda.KdaError):
        kda.gated_norm(torch.zeros(2, 16385, device="cuda"))


def test_graph_and_side_stream(kda):
    x, r, w = c(draw(25, 300, 512, dtype=BF)), c(draw(26, 300, 512, dtype=BF)), c(draw(27, 512))
    ro, y = kda.block_norm(x, r, w, w)
    n = kda.gated_norm(y, w, x, "silu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r3, y3 = kda.block_norm(x, r, w, w, stream=side)
    side.synchronize()
    assert torch.equal(r3, ro) and torch.equal(y3, y)
    r2, y2, n2 = torch.empty_like(ro), torch.empty_like(y), torch.empty_like(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.block_norm(x, r, w, w, residual_out=r2, out=y2)
        kda.gated_norm(y2, w, x, "silu", out=n2)
    for _ in range(3):
        r2.zero_(), y2.zero_(), n2.zero_()
        graph.replay()
        kda.gated_norm(x, w)
        torch.cuda.synchronize()
        assert torch.equal(r2, ro) and torch.equal(y2, y) and torch.equal(n2, n)


def test_offsets_past_32_bits(kda):
    rows, dim = (1 << 31) // 1024 + 5, 1024
    x = torch.ones(rows, dim, dtype=BF, device="cuda")
    tail = draw(28, 9, dim, dtype=BF)
    x[-9:] = tail.cuda()
    y = kda.gated_norm(x)
    check_gated(tail, None, None, None, False, 1e-6, y[-9:])
    ro, _ = kda.block_norm(y, x, residual_out=x)
    got = ro[-9:].cpu()
    ref = host64(tail) + host64(y[-9:])
    assert np.all(np.abs(host64(got) - ref) <= 1.01 * U[BF] * np.abs(ref) + 4 * U32 * np.abs(ref))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [512, 513])
@pytest.mark.parametrize("dim", [300, 768, 1000, 2050, 4096])
def test_wide_rows_many_of_them(kda, dtype, rows, dim):
    """Up to 512 rows a thread takes one vector of a row, beyond that two."""
    x, z = draw(31, rows, dim, dtype=dtype), draw(32, rows, dim, dtype=dtype)
    w, v, r = draw(33, dim), draw(34, dim), draw(35, rows, dim)
    check_gated(x, w, z, "silu", False, 1e-6, kda.gated_norm(c(x), c(w), c(z), "silu"))
    ro, y = kda.block_norm(c(x), c(r), c(w), c(v), c(z), "sigmoid", scale=0.5)
    check_block(x, r, w, v, z, "sigmoid", None, 0.5, 1e-6, ro, y)
    x[3] = float("nan")  # a row of its own
    same = kda.gated_norm(c(x), c(w), c(z), "silu")
    assert torch.isnan(same[3]).all() and torch.isfinite(same[:3]).all() and torch.isfinite(same[4:]).all()
