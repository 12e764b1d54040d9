"""Linear attention with a decay per head on the GPU against the fp64 oracle:
every head dim, type and decay form, lengths from none to several segments,
strided tensors, state pools, values that are not finite, streams and graphs.
Bounds: layer_cases.py."""
import numpy as np
import pytest
import torch

import oracle
from layer_cases import U, check_linear, cuda, host64, linear_inputs, linear_reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def run(kda, d, **kw):
    return kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_prefill_head_dims(kda, dtype, dk, dv):
    i = linear_inputs(1, [70, 0, 1, 129, 300], 4, 2, dk, dv, dtype)
    o, ht = run(kda, cuda(i))
    check_linear(i, o, ht)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127], [255], [256], [257], [700],
                                     [1, 513, 256, 0, 1024], [0, 0, 3], [1] * 40, [5000]])
def test_prefill_lengths(kda, dtype, lengths):
    i = linear_inputs(2, lengths, 2, 1, 64, 64, dtype, g_scale=0.05)
    o, ht = run(kda, cuda(i))
    check_linear(i, o, ht)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("g_scale", [0.0, 1e-3, 1.0, 30.0, 1e6])
def test_prefill_decays(kda, decay, g_scale):
    for dtype in (BF, F32):
        i = linear_inputs(3, [333, 90], 3, 3, 32, 64, dtype, decay=decay, g_scale=g_scale)
        o, ht = run(kda, cuda(i))
        check_linear(i, o, ht)


def test_prefill_strong_decay_among_weak_ones(kda):
    """A decay of e^-200 or of nothing left (-inf) in the middle of a chunk: what
    follows it keeps its digits."""
    for value in (-200.0, -1e4, -float("inf")):
        i = linear_inputs(4, [150], 2, 2, 64, 32, F32, g_scale=0.01)
        for t in (5, 20, 64, 100):
            i["g"][t] = value
        o, ht = run(kda, cuda(i))
        check_linear(i, o, ht)


def test_prefill_without_states(kda):
    i = linear_inputs(5, [100, 600], 2, 2, 64, 64, BF, h0=False)
    d = cuda(i)
    o, ht = run(kda, d)
    check_linear(i, o, ht)
    o2, none = run(kda, d, output_final_state=False, scale=0.25)
    assert none is None
    check_linear(i, o2, None, scale=0.25)
    one = linear_inputs(6, [77], 2, 2, 64, 64, BF, h0=False)
    c = cuda(one)
    check_linear(one, *kda.linear_prefill(c["q"], c["k"], c["v"], c["g"]))


def test_prefill_bf16_states_and_pool(kda):
    """A pool of bf16 states updated in place: skipped sequences (negative or
    past the pool) write nothing, the other slots and rows stay as they were."""
    lengths = [30, 700, 0, 5, 64, 200]
    i = linear_inputs(7, lengths, 2, 1, 64, 128, BF, n_states=9, state_dtype=BF)
    slots = [3, 0, 8, -1, 9, 5]
    d = cuda(i)
    before = d["h0"].clone()
    out = torch.full_like(d["v"], 7.0)
    o, ht = run(kda, d, out=out, state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert ht is d["h0"] and o is out
    cu = np.concatenate([[0], np.cumsum(lengths)])
    used = set()
    for n, s in enumerate(slots):
        rows = slice(int(cu[n]), int(cu[n + 1]))
        if not 0 <= s < 9:
            assert torch.all(out[rows] == 7.0)
            continue
        used.add(s)
        part = {x: i[x][rows] for x in "qkvg"}
        part.update(h0=i["h0"][s:s + 1], cu=torch.tensor([0, lengths[n]], dtype=torch.int32))
        check_linear(part, out[rows], ht[s:s + 1])
    for s in range(9):
        if s not in used:
            assert torch.equal(ht[s], before[s])


@pytest.mark.parametrize("lengths", [[90, 40], [900, 300]])
def test_prefill_in_place_states(kda, lengths):
    i = linear_inputs(8, lengths, 2, 2, 128, 64, BF, g_scale=0.02)
    d = cuda(i)
    o1, h1 = run(kda, d)
    st = d["h0"].clone()
    o2, h2 = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], st, d["cu"], ht=st)
    assert h2 is st and torch.equal(o1, o2) and torch.equal(h1, h2)
    check_linear(i, o2, h2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_slices_of_wider_buffers(kda, dtype):
    """q, k, v as slices of one fused projection and o as a slice of a wider
    buffer whose other columns stay as they were."""
    H, Hk, dk, dv, T = 4, 2, 32, 64, 400
    i = linear_inputs(9, [150, 250], H, Hk, dk, dv, dtype)
    d = cuda(i)
    w = 2 * Hk * dk + H * dv
    fused = torch.cat([d["q"].view(T, -1), d["k"].view(T, -1), d["v"].view(T, -1),
                       torch.zeros(T, 24, dtype=dtype, device="cuda")], 1).contiguous()
    d["q"] = fused[:, :Hk * dk].unflatten(1, (Hk, dk))
    d["k"] = fused[:, Hk * dk:2 * Hk * dk].unflatten(1, (Hk, dk))
    d["v"] = fused[:, 2 * Hk * dk:w].unflatten(1, (H, dv))
    wide = torch.full((T, H * dv + 40), 3.0, dtype=dtype, device="cuda")
    out = wide[:, 16:16 + H * dv].unflatten(1, (H, dv))
    o, ht = run(kda, d, out=out)
    check_linear(i, o, ht)
    assert torch.all(wide[:, :16] == 3.0) and torch.all(wide[:, 16 + H * dv:] == 3.0)


def test_prefill_rows_outside_sequences(kda):
    """Rows before the first and behind the last sequence are left alone, and
    tables that break the rules stay in bounds."""
    i = linear_inputs(10, [40, 60, 20], 2, 2, 32, 32, BF)
    d = cuda(i)
    out = torch.full_like(d["v"], 5.0)
    ragged = dict(i, cu=torch.tensor([10, 40, 100], dtype=torch.int32), h0=i["h0"][:2])
    d2 = dict(d, cu=ragged["cu"].cuda(), h0=d["h0"][:2].contiguous())
    o, ht = run(kda, d2, out=out)
    assert torch.all(out[:10] == 5.0) and torch.all(out[100:] == 5.0)
    ro, rh, ao, ah = linear_reference(ragged)
    part = dict(ragged)
    check_linear(part, o[10:100], ht, ref=(ro[10:100], rh, ao[10:100], ah))
    for table in ([-5, 200, 100, 50], [120, 60, 0, 7], [1 << 30, -(1 << 31), 3, 2147483647]):
        d3 = dict(d, cu=torch.tensor(table, dtype=torch.int32, device="cuda"))
        run(kda, d3)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("where", ["v", "k", "q", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_prefill_nonfinite_values_stay_behind_their_token(kda, dtype, where, value):
    """A value that is not finite at one token and head changes nothing before
    that token, in another head, or in another sequence."""
    if where == "g" and value == -float("inf"):
        pytest.skip("-inf is a decay")
    i = linear_inputs(11, [130, 45], 2, 2, 64, 64, dtype)
    clean = run(kda, cuda(i))
    for t in (0, 21, 50, 100):
        b = dict(i)
        b[where] = i[where].clone()
        if where == "g":
            b[where][t, 1] = value
        else:
            b[where][t, 1, 3] = value
        o, ht = run(kda, cuda(b))
        assert torch.equal(o[:, 0], clean[0][:, 0]) and torch.equal(o[:t], clean[0][:t])
        assert torch.equal(o[130:], clean[0][130:]) and torch.equal(ht[1], clean[1][1])
        assert torch.equal(ht[0, 0], clean[1][0, 0])
        with np.errstate(all="ignore"):
            ro, rh = linear_reference(b)[:2]
        # not finite exactly where the recurrence is not
        assert torch.equal(torch.isfinite(o[:130, 1]).cpu(), torch.from_numpy(np.isfinite(ro[:130, 1])))
        assert torch.equal(torch.isfinite(ht[0, 1]).cpu(), torch.from_numpy(np.isfinite(rh[0, 1])))


@pytest.mark.parametrize("dtype,state", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("N,H,Hk,decay", [(1, 1, 1, "token"), (3, 4, 2, "head"), (150, 4, 1, "token")])
def test_decode(kda, dtype, state, dk, dv, N, H, Hk, decay):
    i = linear_inputs(12, [1] * N, H, Hk, dk, dv, dtype, decay=decay, state_dtype=state)
    d = cuda(i)
    o = kda.linear_decode(d["h0"], d["q"], d["k"], d["v"], d["g"])
    check_linear(i, o, d["h0"])


def test_decode_pool_strides_and_strong_decays(kda):
    N, H, Hk, dk, dv = 6, 4, 2, 64, 32
    i = linear_inputs(13, [1] * N, H, Hk, dk, dv, BF, n_states=8, state_dtype=BF)
    i["g"][0, 1] = -float("inf")
    i["g"][1] = -1e5
    d = cuda(i)
    slots = [7, 2, -3, 0, 8, 4]
    before = d["h0"].clone()
    buf = torch.zeros(N, Hk * dk + 16, dtype=BF, device="cuda")
    buf[:, :Hk * dk] = d["q"].view(N, -1)
    wide = torch.full((N, H * dv + 8), 2.0, dtype=BF, device="cuda")
    out = wide[:, :H * dv].unflatten(1, (H, dv))
    o = kda.linear_decode(d["h0"], buf[:, :Hk * dk].unflatten(1, (Hk, dk)), d["k"], d["v"], d["g"], out=out,
                          scale=0.3, state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    live = [n for n, s in enumerate(slots) if 0 <= s < 8]
    for n in range(N):
        if n not in live:
            assert torch.all(o[n] == 2.0)
            continue
        part = {x: i[x][n:n + 1] for x in "qkvg"}
        part.update(h0=i["h0"][slots[n]:slots[n] + 1], cu=torch.tensor([0, 1], dtype=torch.int32))
        check_linear(part, o[n:n + 1], d["h0"][slots[n]:slots[n] + 1], scale=0.3)
    for s in set(range(8)) - {slots[n] for n in live}:
        assert torch.equal(d["h0"][s], before[s])
    assert torch.all(wide[:, H * dv:] == 2.0)


def test_prefill_then_decode_is_a_longer_prefill(kda):
    i = linear_inputs(14, [260, 33], 2, 2, 128, 128, F32, g_scale=0.1)
    d = cuda(i)
    cut = {x: torch.cat([d[x][:259], d[x][260:292]]).contiguous() for x in "qkvg"}
    last = {x: torch.stack([d[x][259], d[x][292]]) for x in "qkvg"}
    o, ht = kda.linear_prefill(cut["q"], cut["k"], cut["v"], cut["g"], d["h0"],
                               torch.tensor([0, 259, 291], dtype=torch.int32, device="cuda"))
    od = kda.linear_decode(ht, last["q"], last["k"], last["v"], last["g"])
    whole = torch.cat([o[:259], od[:1], o[259:], od[1:]])
    check_linear(i, whole, ht)


def test_empty_calls(kda):
    e = torch.zeros(0, 2, 32, dtype=BF, device="cuda")
    h0 = torch.randn(3, 2, 32, 32, device="cuda")
    o, ht = kda.linear_prefill(e, e, e, torch.zeros(0, 2, device="cuda"), h0,
                               torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, 2, 32) and torch.equal(ht, h0)
    assert kda.linear_decode(torch.zeros(0, 2, 32, 32, device="cuda"), e, e, e,
                             torch.zeros(0, 2, device="cuda")).shape == (0, 2, 32)


def test_wrapper_refusals(kda):
    i = cuda(linear_inputs(15, [20], 2, 2, 32, 32, BF))
    q, k, v, g, h0 = (i[x] for x in ("q", "k", "v", "g", "h0"))
    for bad in (dict(q=q.float()), dict(k=k[:10]), dict(v=v.cpu()), dict(g=g.double()), dict(g=g[:, :1]),
                dict(h0=h0.half()), dict(h0=h0[:, :1]), dict(h0=h0.cpu()),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(cu_seqlens=torch.tensor([0, 20], device="cuda")), dict(state_dtype=BF),
                dict(out=v.float()), dict(ht=h0.bfloat16()), dict(workspace=torch.zeros(4)),
                dict(state_indices=torch.tensor([0], device="cuda"))):
        kw = dict(dict(q=q, k=k, v=v, g=g, h0=h0), **bad)
        with pytest.raises((TypeError, ValueError)):
            kda.linear_prefill(**kw)
    with pytest.raises(kda.KdaError):
        kda.linear_prefill(q, k, v, g, h0, out=q)          # o over q
    with pytest.raises(kda.KdaError):
        kda.linear_decode(h0[:1], q[:1], k[:1], v[:1], g[:1], scale=float("nan"))
    with pytest.raises((TypeError, ValueError)):
        kda.linear_decode(h0[:1], q[:2], k[:2], v[:2], g[:2])


def test_side_stream(kda):
    """A call on a stream that is not the current one, its outputs and workspace
    made for that stream."""
    i = linear_inputs(16, [900], 2, 2, 64, 64, BF, g_scale=0.05)
    d = cuda(i)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    o, ht = run(kda, d, stream=side)
    st = d["h0"].clone()
    torch.cuda.synchronize()
    check_linear(i, o, ht)
    od = kda.linear_decode(st, d["q"][:1], d["k"][:1], d["v"][:1], d["g"][:1], stream=side)
    side.synchronize()
    part = {x: i[x][:1] for x in "qkvg"}
    part.update(h0=i["h0"], cu=torch.tensor([0, 1], dtype=torch.int32))
    check_linear(part, od, st)


def test_two_graphs_replayed(kda):
    """Two captured prefills and a captured decode, replayed in turn with eager
    work between: every replay gives the eager results bit for bit."""
    cases = []
    for seed, lengths in ((17, [700, 0, 333]), (18, [100, 900])):
        d = cuda(linear_inputs(seed, lengths, 4, 2, 128, 64, BF, g_scale=0.05))
        ws = torch.empty(kda.linear_workspace_bytes(sum(lengths), 4, 128, 64, len(lengths)),
                         dtype=torch.uint8, device="cuda")
        o, ht = run(kda, d, workspace=ws)
        st = ht.clone()
        od = kda.linear_decode(st, d["q"][:len(lengths)], d["k"][:len(lengths)], d["v"][:len(lengths)],
                               d["g"][:len(lengths)])
        cases.append(dict(d=d, ws=ws, want=(o.clone(), ht.clone(), od.clone(), st.clone()), n=len(lengths),
                          o=torch.empty_like(o), ht=torch.empty_like(ht), od=torch.empty_like(od)))
    torch.cuda.synchronize()
    for c in cases:
        c["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c["graph"]):
            run(kda, c["d"], out=c["o"], ht=c["ht"], workspace=c["ws"])
            n, d = c["n"], c["d"]
            kda.linear_decode(c["ht"], d["q"][:n], d["k"][:n], d["v"][:n], d["g"][:n], out=c["od"])
    for rep in range(3):
        for c in cases:
            c["o"].fill_(9.0)
            c["ht"].fill_(9.0)
            c["ws"].fill_(255)
        for c in cases:
            c["graph"].replay()
        run(kda, cases[0]["d"])  # eager work of its own between the replays
        torch.cuda.synchronize()
        for c in cases:
            o, _, od, st = c["want"]
            assert torch.equal(c["o"], o) and torch.equal(c["od"], od) and torch.equal(c["ht"], st)


def test_same_bits_every_time(kda):
    d = cuda(linear_inputs(19, [3000, 17], 8, 4, 128, 128, BF, g_scale=0.02))
    o, ht = run(kda, d)
    for _ in range(3):
        o2, h2 = run(kda, d)
        assert torch.equal(o, o2) and torch.equal(ht, h2)


def test_packing_changes_no_bits(kda):
    """A sequence's results do not depend on what it is packed with, as long as
    its segments stay the same."""
    lens = [70, 200, 1, 130]
    i = linear_inputs(20, lens, 2, 2, 64, 64, BF)
    d = cuda(i)
    o, ht = run(kda, d)
    cu = np.concatenate([[0], np.cumsum(lens)])
    for n in range(4):
        s = slice(int(cu[n]), int(cu[n + 1]))
        o1, h1 = kda.linear_prefill(*(d[x][s].contiguous() for x in "qkvg"), h0=d["h0"][n:n + 1].contiguous())
        assert torch.equal(o1, o[s]) and torch.equal(h1[0], ht[n])


def test_offsets_past_32_bits(kda):
    """A prompt of 2^31 and more values per tensor: the last tokens, whose state
    has forgotten the rest (decay e^-2 a token), against the oracle."""
    H, D, T = 32, 128, (1 << 31) // (32 * 128) + 777
    gen = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = (torch.randn(T, H, D, device="cuda", dtype=BF, generator=gen) for _ in range(3))
    g = torch.full((H,), -2.0, device="cuda")
    o, ht = kda.linear_prefill(q, k, v, g)
    n = 60
    part = dict(q=q[-n:].cpu(), k=k[-n:].cpu(), v=v[-n:].cpu(), g=g.cpu(), h0=None,
                cu=torch.tensor([0, n], dtype=torch.int32))
    ro, rh, ao, ah = linear_reference(part)
    # e^-80 of earlier state is left at token n - 20: below every bound
    m = n - 20
    sel = lambda x: x[m:]  # noqa: E731
    check_linear(part, o[-20:], ht, ref=(sel(ro), rh, sel(ao), ah))
    del o, ht, q, k, v
    # a pool whose slots lie past 2^31 values
    S = (1 << 31) // (H * D * D) + 9
    pool = torch.zeros(S, H, D, D, device="cuda", dtype=BF)
    i = linear_inputs(22, [1, 1], H, H, D, D, BF, state_dtype=BF)
    d = cuda(i)
    slots = torch.tensor([S - 1, S - 4], dtype=torch.int32, device="cuda")
    pool[slots.long()] = d["h0"]
    od = kda.linear_decode(pool, d["q"], d["k"], d["v"], d["g"], state_indices=slots)
    check_linear(i, od, pool[slots.long()])
    pool[slots.long()] = d["h0"]
    op, _ = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], pool, d["cu"], state_indices=slots)
    check_linear(i, op, pool[slots.long()])


@pytest.mark.parametrize("n", [64, 65, 200, 1000])
def test_prefill_many_sequences(kda, n):
    """More sequences than lanes, empty and long ones among them."""
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 9, size=n)
    lengths[rng.integers(0, n, size=2)] = (700, 1500)
    i = linear_inputs(23, [int(x) for x in lengths], 2, 2, 32, 32, BF, g_scale=0.1)
    o, ht = run(kda, cuda(i))
    check_linear(i, o, ht)


@pytest.mark.parametrize("H,Hk,dk,dv", [(8, 2, 64, 32), (8, 4, 32, 64), (12, 1, 64, 64), (6, 6, 128, 128), (4, 1, 128, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_heads_sharing_a_key_head(kda, H, Hk, dk, dv, dtype):
    i = linear_inputs(24, [500, 3, 0, 90], H, Hk, dk, dv, dtype, g_scale=0.2)
    o, ht = run(kda, cuda(i))
    check_linear(i, o, ht)


def test_two_streams_at_once(kda):
    """Calls in flight on two streams, each with a workspace of its own: the
    results of either alone, bit for bit."""
    sets = [cuda(linear_inputs(s, [1500, 700], 4, 4, 128, 128, BF, g_scale=0.05)) for s in (25, 26)]
    want = [run(kda, d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for d, s in zip(sets, streams):
            got.append(run(kda, d, stream=s))
        torch.cuda.synchronize()
        for (o, ht), (wo, wh) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(ht, wh)


def test_pools_given_one_way_only(kda):
    """A pool to read from without one to write to, and the reverse."""
    i = linear_inputs(27, [20, 150], 2, 2, 32, 64, BF, n_states=4)
    d = cuda(i)
    idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    part = dict(i, h0=i["h0"][[3, 1]].contiguous())
    before = d["h0"].clone()
    o, none = run(kda, d, state_indices=idx, output_final_state=False)
    assert none is None and torch.equal(d["h0"], before)
    check_linear(part, o, None)
    pool = torch.full_like(d["h0"], 6.0)
    o, ht = kda.linear_prefill(d["q"], d["k"], d["v"], d["g"], None, d["cu"], ht=pool, state_indices=idx)
    assert ht is pool and torch.all(pool[0] == 6.0) and torch.all(pool[2] == 6.0)
    check_linear(dict(i, h0=None), o, pool[[3, 1]])
    both = torch.full_like(d["h0"], 6.0)
    o, ht = run(kda, d, ht=both, state_indices=idx)
    assert torch.equal(d["h0"], before)
    check_linear(part, o, both[[3, 1]])


@pytest.mark.parametrize("dk,dv,Hk", [(32, 32, 4), (32, 128, 4), (64, 64, 2), (128, 32, 1), (128, 64, 2), (128, 128, 4), (64, 128, 2)])
def test_prefill_few_tokens_per_sequence(kda, dk, dv, Hk):
    """Continuing prefills: at most 64 tokens a sequence on average, one of them longer."""
    i = linear_inputs(28, [1, 31, 32, 33, 0, 64, 65, 127, 5, 2], 4, Hk, dk, dv, BF, state_dtype=BF)
    o, ht = run(kda, cuda(i))
    check_linear(i, o, ht)
    b = dict(i, v=i["v"].clone())
    b["v"][40, 1, 3] = float("inf")  # in the third sequence
    o2, h2 = run(kda, cuda(b))
    assert torch.equal(o2[:40], o[:40]) and torch.equal(o2[64:], o[64:]) and torch.equal(h2[3:], ht[3:])
    assert torch.isinf(o2[40:64, 1, 3]).any() or torch.isnan(o2[40:64, 1, 3]).any()


@pytest.mark.parametrize("H,T", [(1, 700), (2, 4097), (3, 2500)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_joins_of_every_length(kda, H, T, dtype):
    """Few heads: the join's workgroups are a wave, its segments come in runs of 16, 8, 4, 2, 1."""
    i = linear_inputs(29, [T], H, H, 64, 64, dtype)
    check_linear(i, *run(kda, cuda(i)))
