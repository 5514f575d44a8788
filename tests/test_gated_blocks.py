"""The 64-bit block reference of the GPU tests against the token-by-token one (CPU)."""
import numpy as np
import pytest
import torch

from gated_blocks import gradients, norms, worst
from gated_cases import inputs
from oracle import gated

CU = [0, 31, 31, 32, 97, 170]


@pytest.mark.parametrize("kind", ["mixed", "mild", "reset", "grow", "none"])
@pytest.mark.parametrize("states", [False, True])
def test_it_is_the_recurrence(kind, states):
    x = inputs(CU, 3, 64, torch.float32, 71, "cpu", kind=kind, grad=True, states=states)
    got = gradients(x, CU)
    o, last = gated.prefill(x["q"], x["k"], x["v"], x["g"], CU, x.get("initial"))
    ref = gated.backward(x["q"], x["k"], x["v"], x["g"], x["do"], CU, x.get("initial"), x.get("d_state"))
    for n, r in zip(("o", "state", "dq", "dk", "dv", "dg", "d_initial"), (o, last) + ref):
        # sums of some thousand 64-bit terms
        np.testing.assert_allclose(got[n].numpy(), r, rtol=1e-10, atol=1e-11, err_msg=n)
    assert bool((got["size"] >= 0).all())


def test_errors_are_per_sequence_and_head():
    ref = torch.ones(10, 2, 4)
    got = ref.clone()
    got[9, 1] = 1.5                       # the only token of the last sequence, one head
    assert worst(got, ref, [0, 9, 9, 10]) == pytest.approx(0.5)
    assert norms(ref, [0, 9, 9, 10]).tolist() == [[6.0, 6.0], [0.0, 0.0], [2.0, 2.0]]
    assert worst(ref, ref, [0, 9, 9, 10]) == 0.0
