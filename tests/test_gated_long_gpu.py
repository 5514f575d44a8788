"""Gated calls whose kernels run through many blocks, segments and tiles, each sequence and head
on its own against the 64-bit block reference.

The chains: the prefill kernel and the two state scans go through rings of two and three slots,
the gradient kernel through several tiles per CTA.  A short chain ends before a slot is used for
the third time.

Tolerances, relative 2-norm of one sequence and head.  bf16 o, dv: one rounding of P or of the
state's snapshot, one of the result, each at most 2^-8 of its value: 2 * 2^-8.  dq, dk: the same
with dP and the result.  (The terms that are rounded have independent errors, and their sum is a
vector of D entries, whose norm does not cancel.)  Over 64 and more tokens the roundings are many
and independent, each uniform within half a step of at most 2^-8 of the value: root mean square
2^-8 / sqrt(3), two of them sqrt(2 / 3) * 2^-8.  States and fp32 results: sums of fp32 terms in
blocks, below 2^-24 * sqrt(terms) of the terms' root sum of squares; 1e-5 as elsewhere.
"""
import ctypes

import numpy as np
import pytest
import torch

from gated_blocks import gradients, norms, worst
from gated_cases import HALF_STEP, inputs
from long_context_04_b200 import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
KINDS = [(BF, 64), (BF, 128), (F32, 64), (F32, 128)]
IDS = ["bf16-d64", "bf16-d128", "fp32-d64", "fp32-d128"]


def bounds(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def ok():
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK


def forward(x, cu):
    return api.gated_prefill(*(x[n] for n in "qkvg"), cu_seqlens=cu, initial_state=x.get("initial"),
                             return_state=True)


def backward(x, cu):
    return api.gated_prefill_backward(*(x[n] for n in "qkvg"), x["do"], cu_seqlens=cu,
                                      initial_state=x.get("initial"), d_state=x.get("d_state"))


def check(x, cu, dtype):
    tol = 2 * HALF_STEP[BF] if dtype == BF else 1e-5
    o, st = forward(x, cu)
    got = backward(x, cu)
    ok()
    ref = gradients(x, cu)
    assert worst(o, ref["o"], cu) <= tol
    assert worst(st, ref["state"], None) <= 1e-5
    for y, n in zip(got, ("dq", "dk", "dv")):
        assert worst(y, ref[n], cu) <= tol, n
    if dtype == BF:
        for y, n in zip((o,) + tuple(got), ("o", "dq", "dk", "dv")):
            off, norm = norms(y.double() - ref[n], cu), norms(ref[n], cu)
            for s, (a, b) in enumerate(zip(cu, cu[1:])):
                assert b - a < 64 or bool((off[s] <= (2 / 3) ** 0.5 * 2.0 ** -8 * norm[s]).all()), (n, s)
    # dg: what cancels (derived in test_gated_precision_gpu.py; fp32 calls hold the states in 24
    # bits), and what each of its terms is off by itself.  bf16: the result's rounding, 2^-8.  fp32:
    # a pair's share is the product of two sums of D <= 128 terms, each off by 2^-24 of the running
    # sum a term (2 * sqrt(128) * 2^-24 = 1.4e-6, independent roundings), and of an exponential whose
    # argument, up to 16 in absolute value where the weight is above 2^-23, is rounded by 2^-24 of
    # itself (1e-6); then sums over at most 64 tokens, two of them running ones (2 * 64 * 2^-24 =
    # 7.6e-6 of the largest).  Together 1e-5.
    own, held = (2.0 ** -8, 2.0 ** -12) if dtype == BF else (1e-5, 1e-5)
    off = norms(got[3].double() - ref["dg"], cu)
    assert bool((off <= own * norms(ref["dg"], cu) + held * norms(ref["size"], cu) + 1e-30).all())
    if "initial" in x:
        assert worst(got[4], ref["d_initial"], None) <= 1e-5
    return (o, st) + tuple(got)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("states", [False, True], ids=["fresh", "states"])
def test_one_chain(dtype, D, states):
    """So many heads that nothing is cut: chains of 33 and of 17 blocks."""
    H = 40 if D == 128 else 80
    cu = bounds([4097, 2100])
    check(inputs(cu, H, D, dtype, 101, "cuda", grad=True, states=states), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_segments(dtype, D):
    """Few heads, cut into segments; decays from hundreds of tokens to less than one."""
    cu = bounds([15000, 1, 3001])
    check(inputs(cu, 4, D, dtype, 102, "cuda", grad=True, states=True), cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_many_tiles(dtype, D):
    """Several hundred (block, head) tiles of full and partial blocks in any order."""
    lengths = [129, 1, 700, 256, 0, 383, 64, 1000, 2, 511]
    cu = bounds(lengths)
    check(inputs(cu, 48, D, dtype, 103, "cuda", grad=True, states=True), cu, dtype)


@pytest.mark.parametrize("kind", ["mild", "reset", "grow"])
def test_gates(kind):
    cu = bounds([2300, 900])
    check(inputs(cu, 20, 128, BF, 104, "cuda", kind=kind, grad=True, states=True), cu, BF)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("B,N,H", [(2, 5000, 1), (3, 4100, 2), (2, 700, 2)], ids=["two", "three", "joined"])
def test_uniform_batches_in_segments(dtype, D, B, N, H):
    """A uniform batch cut into segments, bit for bit the same sequences packed."""
    cu = [N * i for i in range(B + 1)]
    x = inputs(cu, H, D, dtype, 105, "cuda", kind="mild", grad=True, states=True)
    packed = check(x, cu, dtype)
    y = {n: t if n in ("initial", "d_state") else t.view(B, N, *t.shape[1:]) for n, t in x.items()}
    uniform = forward(y, None) + tuple(backward(y, None))
    ok()
    for a, b in zip(packed, uniform):
        assert torch.equal(a, b.view(a.shape))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_repeats(dtype):
    """Equal inputs, equal bits, over many blocks; and two calls at once on two streams."""
    cu = bounds([3000, 700])
    xs = [inputs(cu, 24, 128, dtype, 106 + i, "cuda", grad=True, states=True) for i in range(2)]
    want = [forward(x, cu) + tuple(backward(x, cu)) for x in xs]
    ok()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = []
        for x, s in zip(xs, sides):
            with torch.cuda.stream(s):
                got.append(forward(x, cu) + tuple(backward(x, cu)))
        ok()
        for a, b in zip(want, got):
            assert all(torch.equal(y, z) for y, z in zip(a, b))


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
def test_every_sequence_by_itself(dtype, D):
    """Short and long sequences of one call, each held to the bounds alone."""
    cu = bounds([300, 0, 1, 129, 64, 2, 17, 1])
    for kind in ("mixed", "steep"):
        check(inputs(cu, 8, D, dtype, 108, "cuda", kind=kind, grad=True, states=True), cu, dtype)
        x = inputs(cu, 8, D, dtype, 109, "cuda", kind=kind, grad=True)
        check(x, cu, dtype)


@pytest.mark.parametrize("dtype,D", KINDS, ids=IDS)
@pytest.mark.parametrize("H,lengths", [(3, [6000, 0, 1, 130]), (48, [1300, 1, 700])], ids=["segments", "chains"])
def test_workspace_is_not_read(dtype, D, H, lengths):
    """A workspace full of NaN, exactly as large as asked for, between guards: the same bits, and
    nothing written beside it."""
    cu = bounds(lengths)
    x = inputs(cu, H, D, dtype, 110, "cuda", grad=True, states=True)
    want = forward(x, cu) + tuple(backward(x, cu))
    L, flags, c = api.lib(), api.LA_BF16 if dtype == BF else api.LA_FP32, np.asarray(cu, np.int32)
    shape = (1, H, cu[-1], D, c.ctypes.data, len(lengths), flags)
    got = [torch.full_like(t, float("nan")) for t in want]
    p = {n: t.data_ptr() for n, t in x.items()}
    for back in (0, 1):
        n = ctypes.c_ulonglong()
        assert L.la_gated_workspace(*shape, back, ctypes.byref(n)) == api.LA_OK
        ws = torch.full((n.value + 2048,), 255, dtype=torch.uint8, device="cuda")
        at = ws.data_ptr() + 1024
        if back:
            o = [t.data_ptr() for t in got[2:]]
            rc = L.la_gated_prefill_backward(p["q"], p["k"], p["v"], p["g"], p["do"], *o[:4], *shape, p["initial"],
                                             p["d_state"], o[4], at, n.value, torch.cuda.current_stream().cuda_stream)
        else:
            rc = L.la_gated_prefill(p["q"], p["k"], p["v"], p["g"], got[0].data_ptr(), *shape, p["initial"],
                                    got[1].data_ptr(), at, n.value, torch.cuda.current_stream().cuda_stream)
        assert rc == api.LA_OK
        ok()
        assert bool((ws[:1024] == 255).all()) and bool((ws[1024 + n.value:] == 255).all())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["initial", "d_state", "neither"])
def test_many_tiles_of_single_blocks(D, which):
    """Sequences of one block, several tiles per CTA, with a state at one end or at none."""
    cu = bounds([100, 128, 31, 77] * 15)
    x = inputs(cu, 9, D, BF, 113, "cuda", kind="mild", grad=True, states=True)
    for n in ("initial", "d_state"):
        if n != which:
            del x[n]
    got = backward(x, cu)
    ok()
    ref = gradients(x, cu)
    for y, n in zip(got, ("dq", "dk", "dv")):
        assert worst(y, ref[n], cu) <= 2 * HALF_STEP[BF], n
    off = norms(got[3].double() - ref["dg"], cu)
    # without states the pairs of the block alone, fp32 sums as above
    own = 2.0 ** -8 + 1e-5
    assert bool((off <= own * norms(ref["dg"], cu) + 2.0 ** -12 * norms(ref["size"], cu)).all())
    if which == "initial":
        assert worst(got[4], ref["d_initial"], None) <= 1e-5
