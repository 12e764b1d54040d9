"""Errors of other HIP calls and the layer calls: what an earlier call of the
thread left behind neither fails a call nor makes it run twice."""
import ctypes

import pytest
import torch

from layer_cases import cuda, linear_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


@pytest.fixture
def older_error():
    """Functions that leave an error in this thread (a refused hipSetDevice, which
    changes nothing) and that take it away again."""
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipGetLastError()

    def leave():
        assert hip.hipSetDevice(1 << 20) != 0

    yield leave, hip.hipGetLastError
    hip.hipGetLastError()


@pytest.mark.parametrize("native", [True, False])
def test_in_place_calls_run_once(kda, older_error, monkeypatch, native):
    from gated_delta_rule_55_amd import layer

    if not native:
        monkeypatch.setattr(layer, "_fast", None)
    d = cuda(linear_inputs(51, [1, 1], 4, 2, 64, 64, BF))
    x, r = torch.randn(7, 256, device="cuda").to(BF), torch.randn(7, 256, device="cuda").to(BF)
    w, w2, o = torch.ones(256, device="cuda"), torch.full((256,), 2.0, device="cuda"), torch.empty_like(d["v"])
    for call, state in (
            (lambda s: kda.linear_decode(s, d["q"], d["k"], d["v"], d["g"], out=o), d["h0"]),
            (lambda s: kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], s, d["cu"], ht=s, out=o), d["h0"]),
            (lambda s: kda.gated_norm(s, w2, x, "sigmoid", out=s), r),
            (lambda s: kda.block_norm(x, s, w, residual_out=s), r)):
        want, got = state.clone(), state.clone()
        call(want)
        torch.cuda.synchronize()
        leave, take = older_error
        leave()  # (torch's own kernels would report it: none runs until it is taken)
        call(got)
        assert take() == 101  # hipErrorInvalidDevice, still there for whoever looks
        torch.cuda.synchronize()
        assert torch.equal(got, want) and not torch.equal(got, state)
