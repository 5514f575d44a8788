"""Gated calls whose tensors have more than 2^31 elements: the last tokens of a long sequence and a
far slot of a large pool, against the 64-bit reference from the state before them."""
import pytest
import torch

from gated_blocks import gradients, norms, worst
from gated_cases import inputs
from long_context_04_b200 import api
from oracle import gated

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,H", [(BF, 64), (F32, 512)], ids=["bf16", "fp32"])
def test_far_tokens(dtype, H):
    D = 128
    T = 2 ** 31 // (H * D) + 301
    tail = 300
    gen = torch.Generator(device="cuda").manual_seed(111)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    x = {n: normal(T, H, D, scale=D ** -0.5) for n in "qkv"}
    x["g"] = torch.rand(T, H, generator=gen, device="cuda").mul_(-0.05).to(dtype)
    assert x["q"].numel() > 2 ** 31
    o, st = api.gated_prefill(*(x[n] for n in "qkvg"), return_state=True)
    _, mid = api.gated_prefill(*(x[n][:T - tail] for n in "qkvg"), return_state=True)
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    heads = [0, 1, H // 2, H - 1]
    y = {n: x[n][T - tail:, heads].contiguous() for n in "qkvg"}
    y["initial"] = mid[:, heads].contiguous()
    y["do"], y["d_state"] = torch.zeros_like(y["q"]), torch.zeros_like(y["initial"])
    ref, cu = gradients(y, [0, tail]), [0, tail]
    tol = 2.0 ** -7 if dtype == BF else 1e-5    # two roundings; fp32 as elsewhere
    assert worst(o[T - tail:, heads], ref["o"], cu) <= tol
    assert worst(st[:, heads], ref["state"], None) <= 2e-5   # the middle state's 1e-5 and its own
    del o
    do = torch.zeros_like(x["q"])
    do[T - tail:].copy_(normal(tail, H, D))
    d_state = torch.randn(1, H, D, D, generator=gen, device="cuda") / D
    got = api.gated_prefill_backward(*(x[n] for n in "qkvg"), do, d_state=d_state)
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    y["do"], y["d_state"] = do[T - tail:, heads].contiguous(), d_state[:, heads].contiguous()
    ref = gradients(y, cu)
    for t, n in zip(got, ("dq", "dk", "dv")):
        assert worst(t[T - tail:, heads], ref[n], cu) <= (tol if dtype == BF else 2e-5), n
    off = norms(got[3][T - tail:, heads].double() - ref["dg"], cu)
    own, held = (2.0 ** -8, 2.0 ** -12) if dtype == BF else (1e-5, 2e-5)
    assert bool((off <= own * norms(ref["dg"], cu) + held * norms(ref["size"], cu)).all())


def test_far_slots():
    """Slots around and beyond element 2^31 of the pool."""
    H, D = 64, 128
    slots = [2047, 2048, 2060, 5]
    pool = torch.zeros(2061, H, D, D, device="cuda")
    assert pool.numel() > 2 ** 31
    x = inputs([0, 4], H, D, BF, 112, "cuda")
    start = torch.randn(4, H, D, D, generator=torch.Generator().manual_seed(7)).cuda()
    pool[slots] = start
    o = api.gated_decode_step(*(x[n] for n in "qkvg"), pool, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    ref_o, ref_s = gated.decode_step(*(x[n] for n in "qkvg"), start)
    assert worst(o, torch.from_numpy(ref_o).cuda(), [0, 1, 2, 3, 4]) <= 2.0 ** -8 + 1e-5
    assert worst(pool[slots], torch.from_numpy(ref_s).cuda(), None) <= 1e-6
    pool[slots] = 0
    assert not pool.any()
