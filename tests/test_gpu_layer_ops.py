"""A layer's step as a user runs it: the short conv writes q, k, v; linear
attention reads them and carries its state; the gated norm, then the block norm
onto the residual stream.  First a prompt, then a token per sequence.  The
oracle composes the same in fp64 from the stored inputs; the bars are those of
bf16 intermediates (each op rounds its output once: 2^-8 a step, four in a
row), relative L2 1e-2.  The same norms behind the KDA step as well."""
import numpy as np
import pytest
import torch

import oracle
import synth
from kda_cases import rel_l2, to_dev
from layer_cases import host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


@pytest.mark.parametrize("H,d,lengths", [(4, 64, [150, 37]), (2, 128, [600, 1, 0])])
def test_conv_linear_norms_prompt_then_token(kda, H, d, lengths):
    dim, N = 3 * H * d, len(lengths)
    cin = synth.make_conv_inputs(31, [n + 1 for n in lengths], dim, 4, "bf16")
    cu_all = cin.cu_seqlens
    pre = np.concatenate([np.arange(cu_all[n], cu_all[n + 1] - 1) for n in range(N)])
    dec = np.array([cu_all[n + 1] - 1 for n in range(N)])
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = int(cu[-1])
    gen = torch.Generator().manual_seed(32)
    total = int(cu_all[-1])
    g = -torch.nn.functional.softplus(torch.randn(total, H, generator=gen))
    z = torch.randn(total, H, d, generator=gen).bfloat16()
    r = torch.randn(total, H * d, generator=gen)
    w_o, w_post, w_pre = (1 + 0.1 * torch.randn(n, generator=gen) for n in (d, H * d, H * d))

    x, w, b, taps = (to_dev(getattr(cin, a), t) for a, t in (("x", "bf16"), ("weight", "f32"),
                                                              ("bias", "f32"), ("state", "bf16")))
    state = torch.zeros(N, H, d, d, device="cuda")
    W = [t.cuda() for t in (w_o, w_post, w_pre)]

    def norms(o, rows):
        y = kda.gated_norm(o, W[0], z[rows].cuda(), "sigmoid")
        return kda.block_norm(y.view(len(rows), H * d), r[rows].cuda(), W[1], W[2])

    q, k, v = kda.causal_conv1d_fwd(x[torch.from_numpy(pre).cuda()].contiguous(), w, b,
                                    torch.from_numpy(cu).cuda(), taps, taps, split=(H * d,) * 3)
    o, _ = kda.linear_prefill(q.view(T, H, d), k.view(T, H, d), v.view(T, H, d), g[pre].cuda(), state,
                              torch.from_numpy(cu).cuda(), ht=state)
    r1, y1 = norms(o, pre)
    q, k, v = kda.causal_conv1d_update(x[torch.from_numpy(dec).cuda()].contiguous(), w, b, taps,
                                       split=(H * d,) * 3)
    o = kda.linear_decode(state, q.view(N, H, d), k.view(N, H, d), v.view(N, H, d), g[dec].cuda())
    r2, y2 = norms(o, dec)

    f = cin.f64()
    qkv, _ = oracle.causal_conv1d(f["x"], f["weight"], f["bias"], cu_all, f["state"], "silu")
    qkv = qkv.reshape(-1, 3, H, d)
    ro, rs = oracle.linear_attention(qkv[:, 0], qkv[:, 1], qkv[:, 2], host64(g), None, cu_all, d ** -0.5)
    rn = oracle.gated_norm(ro, host64(w_o), host64(z), "sigmoid", False, 1e-6).reshape(total, H * d)
    rr, ry = oracle.block_norm(rn, host64(r), host64(w_post), host64(w_pre), None, None, None, 1.0, 1e-6)
    for got, want in ((r1, rr[pre]), (y1, ry[pre]), (r2, rr[dec]), (y2, ry[dec]), (state, rs)):
        assert rel_l2(host64(got), want) <= 1e-2


def test_norms_after_the_kda_step(kda):
    inp = synth.make_inputs(33, [90, 30], 2, 64, dtype="bf16", gate="kimi", h0_std=0.05)
    q, k, v, beta = (to_dev(getattr(inp, a), "bf16") for a in ("q", "k", "v", "beta"))
    cu = torch.from_numpy(inp.cu_seqlens).cuda()
    o, _ = kda.chunk_prefill(q, k, v, to_dev(inp.g, "f32"), beta, to_dev(inp.h0, "f32"), cu, scale=inp.scale)
    gen = torch.Generator().manual_seed(34)
    z, r = torch.randn(120, 2, 64, generator=gen).bfloat16(), torch.randn(120, 128, generator=gen).bfloat16()
    w = 1 + 0.1 * torch.randn(128, generator=gen)
    y = kda.gated_norm(o, w[:64].cuda(), z.cuda(), "sigmoid")
    r1, y1 = kda.block_norm(y.view(120, 128), r.cuda(), weight_pre=w.cuda())
    f = inp.f64()
    ro, _ = oracle.prefill(f["q"], f["k"], f["v"], f["g"], f["beta"], f["h0"], f["cu_seqlens"], f["scale"])
    rn = oracle.gated_norm(ro, host64(w[:64]), host64(z), "sigmoid", False, 1e-6).reshape(120, 128)
    rr, ry = oracle.block_norm(rn, host64(r), None, host64(w), None, None, None, 1.0, 1e-6)
    assert rel_l2(host64(r1), rr) <= 1e-2 and rel_l2(host64(y1), ry) <= 1e-2
