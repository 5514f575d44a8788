"""Gated lightning attention on the GPU against the fp64 recurrence.

Tolerances (relative 2-norm per head).  A value rounded to bf16 is off by at most 2^-8 of
itself; the fp32 path rounds by 2^-24.
  o, dq, dk, dv (bf16): one rounding of the scores or of the state snapshot before the last
      product, and one of the result: 2 * 2^-8.  (Roundings of one product's terms are
      independent of each other, so the sum is off by no larger a share than its terms.)
  dg (bf16): the snapshots of the state and of its gradient meet in one product, then the
      result is rounded: 3 * 2^-8.
  fp32 results and states: sums of up to a few thousand fp32 terms, each added with an error
      of 2^-24 of the running sum: below 1e-5 as for the ungated operators.
"""
import ctypes

import numpy as np
import pytest
import torch

from gated_cases import HALF_STEP, gates, inputs, rel
from long_context_04_b200 import api
from oracle import gated

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
STATE_TOL = 1e-5
LENGTHS = {
    "one": [1], "two": [2], "b63": [63], "b64": [64], "b65": [65], "b127": [127], "b128": [128], "b129": [129],
    "b257": [257], "ragged": [300, 0, 1, 129, 64, 2], "empties": [0, 0, 5, 0],
}
KINDS = [(d, D) for d in (BF, F32) for D in (64, 128)]
IDS = [f"{'bf16' if d == BF else 'fp32'}-d{D}" for d, D in KINDS]


def out_tol(dtype):
    return 2 * HALF_STEP[BF] if dtype == BF else 1e-5


def dg_tol(dtype):
    return 3 * HALF_STEP[BF] if dtype == BF else 1e-5


def bounds(lengths):
    return [0] + list(np.cumsum(lengths).tolist())


def ok():
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK


def check_forward(x, cu, dtype, **kw):
    o, st = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, return_state=True,
                              initial_state=x.get("initial"), **kw)
    ok()
    ref_o, ref_s = gated.prefill(x["q"], x["k"], x["v"], x["g"], cu, x.get("initial"))
    assert rel(o, ref_o) <= out_tol(dtype)
    assert rel(st, ref_s) <= STATE_TOL
    return o, st


def check_backward(x, cu, dtype):
    got = api.gated_prefill_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu,
                                     initial_state=x.get("initial"), d_state=x.get("d_state"))
    ok()
    ref = gated.backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu, x.get("initial"), x.get("d_state"))
    for y, r, name in zip(got[:3], ref[:3], ("dq", "dk", "dv")):
        assert rel(y, r) <= out_tol(dtype), name
    if x["g"] is None:
        assert got[3] is None
    else:
        assert rel(got[3], ref[3]) <= dg_tol(dtype)
    if "initial" in x:
        assert rel(got[4], ref[4]) <= STATE_TOL
    return got


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("lengths", LENGTHS.values(), ids=LENGTHS.keys())
@pytest.mark.parametrize("states", [False, True], ids=["fresh", "states"])
def test_prefill(dtype, D, lengths, states):
    cu = bounds(lengths)
    x = inputs(cu, 4, D, dtype, 1, "cuda", states=states)
    o, st = check_forward(x, cu, dtype)
    for s, n in enumerate(lengths):  # a sequence of no tokens keeps its state bit for bit
        if n == 0:
            assert torch.equal(st[s], x["initial"][s] if states else torch.zeros_like(st[s]))


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("kind", ["none", "zero", "mild", "steep", "reset", "grow"])
def test_prefill_gates(dtype, D, kind):
    cu = bounds([200, 131])
    check_forward(inputs(cu, 3, D, dtype, 2, "cuda", kind=kind, states=True), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_prefill_long_and_few_heads(dtype, D):
    """One long sequence beside short ones on one head: the scan is cut into segments."""
    cu = bounds([5, 6000, 0, 130])
    check_forward(inputs(cu, 1, D, dtype, 3, "cuda", kind="mild", states=True), cu, dtype)


def test_prefill_without_gate_is_prefill():
    cu = bounds([300, 129])
    x = inputs(cu, 2, 128, BF, 4, "cuda", kind="none")
    o = api.gated_prefill(x["q"], x["k"], x["v"], None, cu_seqlens=cu)
    ref = api.prefill(x["q"], x["k"], x["v"], cu_seqlens=cu)
    ok()
    # both are within 2 * 2^-8 of the same number
    assert rel(o, ref.double().cpu().numpy()) <= 4 * HALF_STEP[BF]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_prefill_uniform_batch(dtype):
    B, N, H, D = 3, 150, 2, 64
    x = inputs([0, B * N], H, D, dtype, 5, "cuda")
    q, k, v = (x[n].view(B, N, H, D) for n in "qkv")
    o, st = api.gated_prefill(q, k, v, x["g"].view(B, N, H), return_state=True)
    ok()
    ref_o, ref_s = gated.prefill(x["q"], x["k"], x["v"], x["g"], [0, 150, 300, 450])
    assert rel(o.view(-1, H, D), ref_o) <= out_tol(dtype) and rel(st, ref_s) <= STATE_TOL
    packed = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=[0, 150, 300, 450])
    assert torch.equal(packed, o.view(-1, H, D))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_prefill_state_in_place_and_kept(dtype):
    cu = bounds([130, 0, 70])
    x = inputs(cu, 2, 128, dtype, 6, "cuda", states=True)
    kept = x["initial"].clone()
    o, st = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, return_state=True,
                              initial_state=x["initial"])
    ok()
    assert torch.equal(kept, x["initial"])
    o2, st2 = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, initial_state=x["initial"],
                                state_out=x["initial"])
    ok()
    assert st2 is x["initial"] and torch.equal(st, st2) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_prefill_leaves_other_rows(dtype):
    """Rows behind the last sequence of a larger buffer stay as they were."""
    cu = bounds([70, 61])
    x = inputs(cu, 2, 128, dtype, 7, "cuda")
    big = torch.full((cu[-1] + 90, 2, 128), 7.0, dtype=dtype, device="cuda")
    api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, out=big[:cu[-1]])
    ok()
    assert bool((big[cu[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_no_tokens(dtype):
    """Sequences without tokens: states pass through, gradients too, nothing else is touched."""
    q, g = torch.zeros(0, 2, 64, dtype=dtype, device="cuda"), torch.zeros(0, 2, dtype=dtype, device="cuda")
    x = torch.randn(2, 2, 64, 64, device="cuda")
    o, st = api.gated_prefill(q, q, q, g, cu_seqlens=[0, 0, 0], initial_state=x, return_state=True)
    ok()
    assert o.shape == q.shape and torch.equal(st, x)
    assert not api.gated_prefill(q, q, q, g, cu_seqlens=[0, 0, 0], return_state=True)[1].any()
    got = api.gated_prefill_backward(q, q, q, g, q, cu_seqlens=[0, 0, 0], initial_state=x, d_state=2 * x)
    ok()
    assert torch.equal(got[4], 2 * x) and all(t.numel() == 0 for t in got[:4])
    assert not api.gated_prefill_backward(q, q, q, g, q, cu_seqlens=[0, 0, 0], initial_state=x)[4].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_many_short_sequences(dtype):
    """More sequences than a packed call may name, as one uniform batch; and 1024 packed ones."""
    H, D = 1, 64
    x = inputs([0, 1100 * 3], H, D, dtype, 8, "cuda")
    o = api.gated_prefill(*(x[n].view(1100, 3, H, -1) for n in "qkv"), x["g"].view(1100, 3, H))
    ok()
    ref, _ = gated.prefill(x["q"], x["k"], x["v"], x["g"], list(range(0, 3301, 3)))
    assert rel(o.view(-1, H, D), ref) <= out_tol(dtype)
    cu = [0] + [3 * i + 1 for i in range(1024)]  # the first of one token, the others of three
    n = cu[-1]
    p = api.gated_prefill(*(x[k][:n].contiguous() for k in "qkvg"), cu_seqlens=cu)
    ok()
    ref, _ = gated.prefill(*(x[k][:n] for k in "qkvg"), cu)
    assert rel(p, ref) <= out_tol(dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_sequences_of_one_token(dtype, D):
    """They are decode steps, alone or beside longer and empty sequences, states in place or none."""
    lengths = [1, 300, 0, 1, 1, 130]
    cu = bounds(lengths)
    x = inputs(cu, 3, D, dtype, 21, "cuda", states=True)
    o, st = check_forward(x, cu, dtype)
    kept = x["initial"].clone()
    api.gated_prefill(*(x[n] for n in "qkvg"), cu_seqlens=cu, initial_state=kept, return_state=True, state_out=kept)
    ok()
    assert torch.equal(kept, st)
    one = [s for s, n in enumerate(lengths) if n == 1]
    rows = [cu[s] for s in one]
    step = x["initial"][one].contiguous()
    y = api.gated_decode_step(*(x[n][rows].contiguous() for n in "qkvg"), step)
    ok()
    assert torch.equal(y, o[rows]) and torch.equal(step, st[one])
    fresh = {n: x[n] for n in "qkvg"}
    check_forward(fresh, cu, dtype)
    # only such and empty ones, packed and as a uniform batch
    few = {n: x[n][:4].contiguous() for n in "qkvg"}
    a, sa = check_forward(few, [0, 0, 1, 2, 2, 3, 4], dtype)
    b, sb = api.gated_prefill(*(few[n].unsqueeze(1) for n in "qkvg"), return_state=True)
    ok()
    assert torch.equal(b.squeeze(1), a) and torch.equal(sb, sa[[1, 2, 4, 5]])


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("lengths", LENGTHS.values(), ids=LENGTHS.keys())
@pytest.mark.parametrize("states", [False, True], ids=["fresh", "states"])
def test_backward(dtype, D, lengths, states):
    cu = bounds(lengths)
    check_backward(inputs(cu, 4, D, dtype, 11, "cuda", grad=True, states=states), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("kind", ["none", "zero", "mild", "steep", "reset", "grow"])
def test_backward_gates(dtype, D, kind):
    cu = bounds([200, 131])
    check_backward(inputs(cu, 3, D, dtype, 12, "cuda", kind=kind, grad=True, states=True), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_backward_long_and_few_heads(dtype, D):
    cu = bounds([5, 4500, 0, 130])
    check_backward(inputs(cu, 1, D, dtype, 13, "cuda", kind="mild", grad=True, states=True), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("which", ["initial", "d_state"])
def test_backward_with_one_of_the_states(dtype, D, which):
    for lengths in ([100], [200, 0, 60]):
        cu = bounds(lengths)
        x = inputs(cu, 2, D, dtype, 17, "cuda", grad=True, states=True)
        del x["d_state" if which == "initial" else "initial"]
        check_backward(x, cu, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_backward_uniform_batch_and_repeat(dtype):
    B, N, H, D = 3, 150, 2, 128
    x = inputs([0, B * N], H, D, dtype, 14, "cuda", grad=True)
    cu = [0, 150, 300, 450]
    got = check_backward(x, cu, dtype)
    shaped = [x[n].view(B, N, H, D) for n in ("q", "k", "v", "do")]
    again = api.gated_prefill_backward(*shaped[:3], x["g"].view(B, N, H), shaped[3])
    ok()
    for y, z in zip(got, again):
        assert torch.equal(y, z.view(y.shape))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,lengths", [(2, [9, 0, 1, 16]), (2, [40, 3]), (2, [700, 9]), (80, [5, 0, 16, 2])])
def test_backward_state_gradient_in_place(dtype, H, lengths):
    """The gradient of the initial states written over that of the final ones, at the C boundary;
    calls of short sequences, of single blocks and of several."""
    cu = bounds(lengths)
    x = inputs(cu, H, 64, dtype, 24, "cuda", grad=True, states=True)
    want = check_backward(x, cu, dtype)
    flags = api.LA_BF16 if dtype == BF else api.LA_FP32
    c = np.asarray(cu, np.int32)
    n = ctypes.c_ulonglong()
    L = api.lib()
    assert L.la_gated_workspace(1, H, cu[-1], 64, c.ctypes.data, len(lengths), flags, 1, ctypes.byref(n)) == api.LA_OK
    ws = torch.full((max(n.value, 16),), 255, dtype=torch.uint8, device="cuda")
    got = [torch.full_like(t, float("nan")) for t in want[:4]] + [x["d_state"].clone()]
    ptr = [t.data_ptr() for t in got]
    rc = L.la_gated_prefill_backward(*(x[k].data_ptr() for k in ("q", "k", "v", "g", "do")), *ptr[:4], 1, H, cu[-1], 64,
                                     c.ctypes.data, len(lengths), flags, x["initial"].data_ptr(), ptr[4], ptr[4],
                                     ws.data_ptr(), n.value, torch.cuda.current_stream().cuda_stream)
    assert rc == api.LA_OK
    ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("H,lengths", [(9, [3900, 0, 70]), (24, [1408, 1])], ids=["segments", "one chain"])
def test_fp32_states_beyond_the_cache(H, lengths):
    """fp32 calls whose blocks' states are too many to be formed block by block and joined."""
    cu = bounds(lengths)
    x = inputs(cu, H, 128, F32, 23, "cuda", grad=True, states=True)
    check_forward(x, cu, F32)
    check_backward(x, cu, F32)


def test_gradient_against_differences():
    """The backward call against differences of the forward call's outputs (fp32)."""
    cu = bounds([75, 40])
    x = inputs(cu, 2, 64, F32, 15, "cuda", kind="steep", grad=True, states=True)
    got = dict(zip(("q", "k", "v", "g", "initial"),
                   api.gated_prefill_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu,
                                              initial_state=x["initial"], d_state=x["d_state"])))

    def loss(y):
        o, st = api.gated_prefill(y["q"], y["k"], y["v"], y["g"], cu_seqlens=cu, initial_state=y["initial"],
                                  return_state=True)
        return float((o.double() * x["do"].double()).sum() + (st.double() * x["d_state"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(2)
    for n, grad in got.items():
        d = torch.randn(grad.shape, generator=gen, device="cuda")
        h = 2.0 ** -7
        up, down = (loss({**x, n: x[n] + e * d}) for e in (h, -h))
        want, have = (up - down) / (2 * h), float((grad.double() * d.double()).sum())
        # o has about 15000 entries of relative error 1e-6 in losses of size |o||do|: noise of
        # up to 1e-6 * sqrt(15000) * 2 / (2 h) = 0.016; q, k, v and the state enter linearly
        # (no further error), g through e^g: h^2 / 6 of the third derivative, below 2e-4 of it
        assert abs(have - want) <= 0.03 + 1e-3 * abs(want), n


def test_nonfinite_values_stay_in_their_sequence():
    """Infinities and NaN of one sequence reach no other, forward or backward."""
    cu = bounds([100, 70, 130])
    for dtype in (BF, F32):
        for D in (64, 128):
            x = inputs(cu, 2, D, dtype, 16, "cuda", grad=True)
            bad = {n: t.clone() for n, t in x.items()}
            for n, val in (("q", "inf"), ("k", "nan"), ("v", "-inf"), ("do", "inf")):
                bad[n][cu[1]:cu[2]] = float(val)
            bad["g"][cu[1]:cu[2]] = float("nan")
            rows = torch.ones(cu[-1], dtype=torch.bool)
            rows[cu[1]:cu[2]] = False
            res = []
            for y in (x, bad):
                o, st = api.gated_prefill(y["q"], y["k"], y["v"], y["g"], cu_seqlens=cu, return_state=True)
                gr = api.gated_prefill_backward(y["q"], y["k"], y["v"], y["g"], y["do"], cu_seqlens=cu)
                res.append([t[rows] for t in (o,) + gr] + [st[[0, 2]]])
            ok()
            for a, b in zip(*res):
                assert torch.equal(a, b)


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("kind", ["none", "mixed", "reset"])
def test_decode(dtype, D, kind):
    B, H, P = 5, 3, 9
    x = inputs([0, B], H, D, dtype, 21, "cuda", kind=kind)
    pool = torch.randn(P, H, D, D, generator=torch.Generator().manual_seed(3)).cuda()
    slots = torch.tensor([8, 0, 3, 4, 7], dtype=torch.int32, device="cuda")
    before = pool.clone()
    o = api.gated_decode_step(x["q"], x["k"], x["v"], x["g"], pool, slots=slots)
    ok()
    ref_o, ref_s = gated.decode_step(x["q"], x["k"], x["v"], x["g"], before[slots.long()])
    # o: one rounding of the result, after fp32 sums of D terms
    assert rel(o, ref_o) <= (HALF_STEP[BF] if dtype == BF else 1e-5)
    assert rel(pool[slots.long()], ref_s) <= 1e-6
    rest = [i for i in range(P) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])
    own = before[slots.long()].contiguous()
    assert torch.equal(api.gated_decode_step(x["q"], x["k"], x["v"], x["g"], own), o)
    assert torch.equal(own, pool[slots.long()])


def test_decode_padding_repeated_and_foreign_slots():
    B, H, D = 6, 2, 128
    x = inputs([0, B], H, D, BF, 22, "cuda")
    pool = torch.randn(4, H, D, D, generator=torch.Generator().manual_seed(4)).cuda()
    before, out = pool.clone(), torch.full((B, H, D), 7.0, dtype=BF, device="cuda")
    api.gated_decode_step(x["q"], x["k"], x["v"], x["g"], pool, out=out,
                          slots=torch.tensor([2, -1, 1, -1, -1, -1], dtype=torch.int32, device="cuda"))
    ok()                                       # padding is no fault
    assert bool((out[[1, 3, 4, 5]] == 7).all()) and torch.equal(pool[[0, 3]], before[[0, 3]])
    once, out1 = pool.clone(), out.clone()
    pool.copy_(before)
    out.fill_(7.0)
    api.gated_decode_step(x["q"], x["k"], x["v"], x["g"], pool, out=out,
                          slots=torch.tensor([2, 4, 1, 2, -5, 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_ERR_DEVICE_RANGE
    assert api.device_status() == api.LA_OK
    assert torch.equal(pool, once) and torch.equal(out, out1)  # the first row of a slot counts


def test_decode_continues_prefill():
    """Prefill, hand-off to a pool, then tokens one by one: the rows of one long prefill."""
    cu, H, D, more = bounds([90, 61]), 2, 128, 4
    lengths = [94, 65]
    full = bounds(lengths)
    x = inputs(full, H, D, BF, 23, "cuda", kind="mild")
    ref_o, ref_s = gated.prefill(x["q"], x["k"], x["v"], x["g"], full)
    first = torch.cat([torch.arange(full[s], full[s] + n) for s, n in enumerate((90, 61))]).cuda()
    _, st = api.gated_prefill(*(x[n][first].contiguous() for n in "qkvg"), cu_seqlens=cu, return_state=True)
    pool = torch.zeros(5, H, D, D, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    api.state_out(st, pool, slots)
    for t in range(more):
        rows = torch.tensor([full[0] + 90 + t, full[1] + 61 + t]).cuda()
        o = api.gated_decode_step(*(x[n][rows].contiguous() for n in "qkvg"), pool, slots=slots)
        ok()
        assert rel(o, ref_o[rows.cpu().numpy()]) <= out_tol(BF)
    assert rel(pool[[3, 1]], ref_s) <= STATE_TOL


# ------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_two_streams_at_once(dtype):
    cu = bounds([700, 0, 300])
    xs = [inputs(cu, 2, 128, dtype, 31 + i, "cuda", grad=True, states=True) for i in range(2)]

    def call(x, stream=None):
        o, st = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, initial_state=x["initial"],
                                  return_state=True, stream=stream)
        return (o, st) + api.gated_prefill_backward(
            x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, initial_state=x["initial"],
            d_state=x["d_state"], stream=stream)

    want = [call(x) for x in xs]
    ok()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [call(x, s) for x, s in zip(xs, streams)]
        ok()
        for a, b in zip(want, got):
            assert all(torch.equal(y, z) for y, z in zip(a, b))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_capture_and_replay(dtype):
    cu = bounds([700, 0, 300])
    x = inputs(cu, 2, 128, dtype, 41, "cuda", grad=True, states=True)
    tok = inputs([0, 3], 2, 128, dtype, 42, "cuda")
    pool = torch.zeros(3, 2, 128, 128, device="cuda")

    def call():
        o, st = api.gated_prefill(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, initial_state=x["initial"],
                                  return_state=True)
        api.state_out(st, pool)
        one = api.gated_decode_step(tok["q"], tok["k"], tok["v"], tok["g"], pool)
        return (o, st, one) + api.gated_prefill_backward(
            x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, initial_state=x["initial"],
            d_state=x["d_state"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (43, 44):
        fresh = inputs(cu, 2, 128, dtype, seed, "cuda", grad=True, states=True)
        for n, t in fresh.items():
            x[n].copy_(t)
        graph.replay()
        ok()
        for y, z in zip(got, call()):
            assert torch.equal(y, z)
    ok()
