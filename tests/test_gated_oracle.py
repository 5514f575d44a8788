"""The fp64 reference of the gated operators against automatic differentiation, finite
differences and the ungated oracle (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from gated_cases import inputs
from oracle import gated

CU = [0, 9, 9, 10, 31]


def _loss(x, cu, do, d_state):
    """The scalar whose gradients the backward pass gives, by the recurrence in torch fp64."""
    total = 0
    for s in range(len(cu) - 1):
        S = x["initial"][s]
        for t in range(cu[s], cu[s + 1]):
            S = S * x["g"][t].exp()[:, None, None] + x["k"][t][:, :, None] * x["v"][t][:, None, :]
            total = total + (torch.einsum("hx,hxy->hy", x["q"][t], S) * do[t]).sum()
        total = total + (S * d_state[s]).sum()
    return total


def _case():
    x = inputs(CU, 4, 64, torch.float32, 5, "cpu", grad=True, states=True)
    return {n: t.double() for n, t in x.items()}


def test_gradients_match_autograd():
    x = _case()
    leaves = {n: x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "initial")}
    _loss(leaves, CU, x["do"], x["d_state"]).backward()
    got = gated.backward(x["q"], x["k"], x["v"], x["g"], x["do"], CU, x["initial"], x["d_state"])
    for n, y in zip(("q", "k", "v", "g", "initial"), got):
        np.testing.assert_allclose(y, leaves[n].grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "initial"])
def test_gradients_match_differences(name):
    x = _case()
    got = dict(zip(("q", "k", "v", "g", "initial"),
                   gated.backward(x["q"], x["k"], x["v"], x["g"], x["do"], CU, x["initial"], x["d_state"])))
    gen = torch.Generator().manual_seed(1)
    d = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
    h = 1e-5
    up, down = (_loss({**x, name: x[name] + e * d}, CU, x["do"], x["d_state"]).item() for e in (h, -h))
    want = (up - down) / (2 * h)
    # the central difference is off by h^2/6 of the third derivative and by the rounding of
    # the two losses over 2 h: about 1e-9 of the largest term each
    assert abs(float((got[name] * d.numpy()).sum()) - want) <= 1e-6 * max(1.0, abs(want))


def test_without_decay_it_is_the_ungated_oracle():
    x = inputs(CU, 3, 64, torch.float32, 9, "cpu", kind="none", states=True)
    o, last = gated.prefill(x["q"], x["k"], x["v"], None, CU, x["initial"])
    ref_o, ref_s = oracle.recurrent(x["q"], x["k"], x["v"], CU, initial_state=x["initial"].numpy())
    np.testing.assert_allclose(o, ref_o, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(last, ref_s, rtol=1e-12, atol=1e-13)


def test_decode_is_the_next_row_of_prefill():
    x = inputs([0, 12], 4, 64, torch.float32, 3, "cpu", states=True)
    o, _ = gated.prefill(x["q"], x["k"], x["v"], x["g"], [0, 12], x["initial"])
    _, S = gated.prefill(x["q"][:11], x["k"][:11], x["v"][:11], x["g"][:11], [0, 11], x["initial"])
    od, _ = gated.decode_step(x["q"][11:], x["k"][11:], x["v"][11:], x["g"][11:], S)
    np.testing.assert_allclose(od[0], o[11], rtol=1e-12, atol=1e-14)
