"""The layer calls on a stream of the caller's: their inputs are filled on that
stream, behind a delay, so that a launch on any other stream meets the filler
that stood there before.  Once through the stream argument (the call is made in
Python) and once with the stream as torch's current one (the native module)."""
import contextlib

import pytest
import torch

from layer_cases import check_linear, cuda, linear_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def draw(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def cases():
    """name -> (inputs, call on such inputs and the stream argument)."""
    i = linear_inputs(61, [900, 300], 4, 2, 128, 64, BF, g_scale=0.05)  # split into segments
    d = cuda(i)
    yield "prefill", d, lambda kda, t, kw: kda.linear_prefill(t["q"], t["k"], t["v"], t["g"], t["h0"], t["cu"], **kw)
    j = cuda(linear_inputs(62, [1] * 5, 4, 2, 64, 64, BF))
    yield "decode", j, lambda kda, t, kw: (kda.linear_decode(t["h0"], t["q"], t["k"], t["v"], t["g"], **kw), t["h0"])
    n = dict(x=draw(63, 300, 512), z=draw(64, 300, 512), r=draw(65, 300, 512), w=draw(66, 512, dtype=torch.float32))
    yield "gated", n, lambda kda, t, kw: (kda.gated_norm(t["x"], t["w"], t["z"], "silu", **kw),)
    yield "block", n, lambda kda, t, kw: kda.block_norm(t["x"], t["r"], t["w"], t["w"], t["z"], "sigmoid", **kw)


@pytest.mark.parametrize("how", ["argument", "current"])
@pytest.mark.parametrize("name", ["prefill", "decode", "gated", "block"])
def test_calls_run_on_their_stream(kda, name, how):
    given, call = next((d, f) for n, d, f in cases() if n == name)
    want = [x.clone() for x in call(kda, {a: x.clone() for a, x in given.items()}, {})]
    # what a launch that does not wait would read: NaN, and tables of no tokens
    tensors = {a: torch.zeros_like(x) if x.dtype == torch.int32 else torch.full_like(x, float("nan"))
               for a, x in given.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # some 20 ms
        for a, x in given.items():
            tensors[a].copy_(x)
    with torch.cuda.stream(side) if how == "current" else contextlib.nullcontext():
        got = call(kda, tensors, {} if how == "current" else dict(stream=side))
    assert not side.query()  # the delay lasted past the call
    side.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_the_same_bits_are_right(kda):
    """The eager results that the others are compared with."""
    i = linear_inputs(61, [900, 300], 4, 2, 128, 64, BF, g_scale=0.05)
    d = cuda(i)
    check_linear(i, *kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"]))
