"""The gradient of the log-decays in bf16 calls, sequence by sequence and head by head.

dg is one number per token and head, a sum of terms of either sign: e^{G_C} <dS, S>, shared by all
tokens of a block, and running sums of q_i . (e^{G_i} S do_i) and k_j . (e^{G_C - G_j} dS v_j).
Where these cancel, what is left shows every bit that S and dS were held in, and a norm over many
heads hides it.

Bound, per sequence and head: the result's own rounding, at most 2^-8 of each value, hence of
their norm; and states held to at least 16 bits, two bf16 parts (2^-8 of 2^-8).  The roundings of
a state's elements are independent, so a sum of products with them is off by 2^-16 / sqrt(3) of the
root of the sum of their squares, `size`, as one standard deviation; three such sums, taken at
three standard deviations: 3 * sqrt(3) * 2^-16 / sqrt(3) < 2^-14.  fp32 sums add 2^-24 of terms no
larger, sqrt(D^2 * 128) of them at most: 2^-24 * 2^10.5 < 2^-13.  Together below 2^-12 of `size`.
"""
import pytest
import torch

from gated_blocks import gradients, norms
from gated_cases import inputs
from long_context_04_b200 import api

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def check(x, cu):
    got = api.gated_prefill_backward(*(x[n] for n in "qkvg"), x["do"], cu_seqlens=cu, initial_state=x.get("initial"),
                                     d_state=x.get("d_state"))
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    ref = gradients(x, cu)
    off = norms(got[3].double() - ref["dg"], cu)
    bound = 2.0 ** -8 * norms(ref["dg"], cu) + 2.0 ** -12 * norms(ref["size"], cu)
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("states", [False, True], ids=["fresh", "states"])
@pytest.mark.parametrize("lengths", [[17] * 24, [300, 17, 2, 150, 17, 1, 260, 64, 700], [1500, 9], [16, 5, 11]],
                         ids=["short", "ragged", "long", "shortest"])
def test_gate_gradient(D, states, lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    for seed in range(4):
        x = inputs(cu, 16, D, BF, 80 + seed, "cuda", kind="mild", grad=True, states=states)
        check(x, cu)


@pytest.mark.parametrize("D", [64, 128])
def test_gate_gradient_does_not_depend_on_the_neighbours(D):
    """A short sequence alone, and packed beside a long one: the same bound."""
    for seed in range(4):
        x = inputs([0, 17, 1017], 8, D, BF, 90 + seed, "cuda", kind="mild", grad=True, states=True)
        check(x, [0, 17, 1017])
        alone = {n: (t[:1] if n in ("initial", "d_state") else t[:17]).contiguous() for n, t in x.items()}
        check(alone, [0, 17])
