"""Every instance of the prefill kernel on the GPU, by name of what chooses it:
head dims, heads a workgroup (1, 2 or 4 of one key head), type, chunk length and
whether sequences are split.  test_layer_launches_host.py checks on the host that
these sizes enqueue these instances."""
import numpy as np
import pytest
import torch

import oracle
from layer_cases import check_linear, cuda, host64, linear_inputs, linear_reference
from linear_kernel_cases import DIMS, KINDS, lengths_of

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("dk,dv,H,Hk", DIMS)
def test_instances(kda, dk, dv, H, Hk, dtype, kind):
    lengths = lengths_of(dtype, kind, H)
    bf16_states = dtype == "bf16" and dk != 64
    i = linear_inputs(71, lengths, H, Hk, dk, dv, DT[dtype], g_scale=0.1,
                      state_dtype=torch.bfloat16 if bf16_states else torch.float32)
    need = kda.linear_workspace_bytes(sum(lengths), H, dk, dv, len(lengths), DT[dtype])
    assert (need > 0) == (kind == "split")
    d = cuda(i)
    o, ht = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"])
    check_linear(i, o, ht)


@pytest.mark.parametrize("value,places", [(float("inf"), (2, 19)), (float("nan"), (11, 30))])
@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("dk,dv,H,Hk", DIMS)
def test_instances_with_values_that_are_not_finite(kda, dk, dv, H, Hk, dtype, kind, value, places):
    """In v, at tokens of different halves of a chunk: what is not finite, and
    every bit of what comes before, of other heads and of other sequences."""
    lengths = lengths_of(dtype, kind, H)
    i = linear_inputs(72, lengths, H, Hk, dk, dv, DT[dtype], g_scale=0.1)
    d = cuda(i)
    clean = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"])
    n = int(np.argmax(lengths))
    begin, end = int(sum(lengths[:n])), int(sum(lengths[:n + 1]))
    h, c = H - 1, dv - 3
    heads = [x for x in range(H) if x != h]
    seqs = [x for x in range(len(lengths)) if x != n]
    for at in places:
        t = begin + at
        v = i["v"].clone()
        v[t, h, c] = value
        o, ht = kda.linear_prefill(d["q"], d["k"], v.cuda(), d["g"], d["h0"], d["cu"])
        assert torch.equal(o[:t], clean[0][:t]) and torch.equal(o[end:], clean[0][end:])
        assert torch.equal(o[:, heads], clean[0][:, heads]) and torch.equal(ht[:, heads], clean[1][:, heads])
        assert torch.equal(ht[seqs], clean[1][seqs])
        part = [host64(x[begin:end]) for x in (i["q"], i["k"], v, i["g"])]
        with np.errstate(all="ignore"):
            ro, rh = oracle.linear_attention(*part, host64(i["h0"][n:n + 1]), [0, end - begin], dk ** -0.5)
        assert torch.equal(torch.isfinite(o[begin:end]).cpu(), torch.from_numpy(np.isfinite(ro)))
        assert torch.equal(torch.isfinite(ht[n]).cpu(), torch.from_numpy(np.isfinite(rh[0])))


@pytest.mark.parametrize("dk,dv,H,Hk", DIMS)
def test_short_sequences_of_a_full_batch(kda, dk, dv, H, Hk):
    """More sequences than lanes in chunks of 32, on a pool of bf16 states with
    rows that hold no sequence."""
    N = -(-256 // H) + 9
    lengths = [(n * 7) % 13 for n in range(N)]
    lengths[N // 2] = 100
    assert N > 64 and kda.linear_workspace_bytes(sum(lengths), H, dk, dv, N) == 0
    i = linear_inputs(73, lengths, H, Hk, dk, dv, DT["bf16"], state_dtype=DT["bf16"], g_scale=0.3)
    d = cuda(i)
    slots = torch.arange(N, dtype=torch.int32)
    slots[3], slots[N - 2] = -1, N + 5
    out = torch.full_like(d["v"], 4.0)
    o, ht = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], out=out, state_indices=slots.cuda())
    ro, rh, ao, ah = linear_reference(i)
    cu = i["cu"].numpy()
    live = [n for n in range(N) if n not in (3, N - 2)]
    rows = np.concatenate([np.arange(cu[n], cu[n + 1]) for n in live])
    check_linear(i, o[rows], ht[live], ref=(ro[rows], rh[live], ao[rows], ah[live]))
    for n in (3, N - 2):
        assert torch.all(out[cu[n]:cu[n + 1]] == 4.0) and torch.equal(ht[n].cpu(), i["h0"][n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[700, 40, 0, 333, 51, 64], [9, 33, 64, 0, 50, 40], [30] * 3 + [45] * 40 + [0, 400] * 12])
def test_order_of_the_batch_changes_no_bits(kda, dtype, lengths):
    """Sequences in another order, and beside other sequences of the same number
    and total length: the same bits, in every chunk length and split or not."""
    i = linear_inputs(74, lengths, 4, 2, 64, 64, DT[dtype], g_scale=0.1)
    d = cuda(i)
    o, ht = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"])
    cu = i["cu"].numpy()
    rng = np.random.default_rng(75)
    for order in (np.arange(len(lengths))[::-1], rng.permutation(len(lengths))):
        rows = torch.from_numpy(np.concatenate([np.arange(cu[n], cu[n + 1]) for n in order])).cuda()
        at = torch.from_numpy(order.copy()).cuda()
        cu2 = torch.tensor([0] + [lengths[n] for n in order]).cumsum(0).to(torch.int32).cuda()
        o2, ht2 = kda.linear_prefill(*(d[x][rows].contiguous() for x in "qkvg"), d["h0"][at].contiguous(), cu2)
        assert torch.equal(o2, o[rows]) and torch.equal(ht2, ht[at])
    # one sequence kept, the others replaced and cut differently
    n = int(np.argmax(lengths))
    other = linear_inputs(76, lengths, 4, 2, 64, 64, DT[dtype], g_scale=0.1)
    rest = [x for x in lengths]
    del rest[n]
    total, cuts = sum(rest), np.sort(rng.integers(0, sum(rest) + 1, size=len(rest) - 1))
    cut = np.diff(np.concatenate([[0], cuts, [total]]))
    new = [int(x) for x in cut[:2]] + [lengths[n]] + [int(x) for x in cut[2:]]
    begin = int(sum(new[:2]))
    m = cuda(other)
    for x in "qkvg":
        m[x][begin:begin + lengths[n]] = d[x][cu[n]:cu[n + 1]]
    m["h0"][2] = d["h0"][n]
    cu2 = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    o2, ht2 = kda.linear_prefill(m["q"], m["k"], m["v"], m["g"], m["h0"], cu2)
    assert torch.equal(o2[begin:begin + lengths[n]], o[cu[n]:cu[n + 1]]) and torch.equal(ht2[2], ht[n])


@pytest.mark.parametrize("beside", [[], [500], [64] * 30])
def test_a_sequence_alone_and_in_larger_batches(kda, beside):
    """33 to 64 tokens: in chunks of 32 or 64, within the bounds either way."""
    for n in (33, 50, 64):
        i = linear_inputs(77, [n] + beside, 2, 2, 64, 64, DT["bf16"])
        d = cuda(i)
        check_linear(i, *kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"]))
