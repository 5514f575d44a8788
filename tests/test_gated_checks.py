"""Argument checks of the gated operators, binding and C ABI (CPU: nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_04_b200 import api, build

FAKE = 0x10000  # aligned and never dereferenced: the checks come first


class Reached(Exception):
    pass


@pytest.fixture
def stub(monkeypatch):
    monkeypatch.setattr(api, "_on_gpu", lambda t: True)

    def reached():
        raise Reached()
    monkeypatch.setattr(api, "lib", reached)


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def test_prefill_binding(stub):
    q, g = bf(10, 2, 64), bf(10, 2)
    for kw in (dict(), dict(cu_seqlens=[0, 4, 10], state_out=f32(2, 2, 64, 64)), dict(out=bf(10, 2, 64)),
               dict(initial_state=f32(1, 2, 64, 64))):
        with pytest.raises(Reached):
            api.gated_prefill(q, bf(10, 2, 64), q, g, **kw)
    with pytest.raises(Reached):
        api.gated_prefill(q, q, q, None)
    q4 = bf(2, 5, 2, 64)
    with pytest.raises(Reached):
        api.gated_prefill(q4, q4, q4, bf(2, 5, 2))
    pool = f32(3, 2, 64, 64)
    for args, kw, text in [
        ((q, bf(10, 2, 128), q, g), {}, "one shape"),
        ((q, q, q, f32(10, 2)), {}, "g must be"),
        ((q, q, q, bf(10, 3)), {}, "g must have shape"),
        ((q, q, q, bf(10, 2, 1)), {}, "g must have shape"),
        ((q, q, q, bf(10, 4)[:, ::2]), {}, "contiguous"),
        ((q4, q4, q4, bf(2, 5, 2)), dict(cu_seqlens=[0, 10]), "cu_seqlens"),
        ((q, q, q, g), dict(out=bf(9, 2, 64)), "out must have shape"),
        ((q, q, q, g), dict(out=q), "overlap"),
        ((q, q, q, g), dict(state_out=f32(2, 2, 64, 64)), "state_out must have shape"),
        ((q, q, q, g), dict(initial_state=f32(2, 2, 64, 64)), "initial_state must have shape"),
        ((q, q, q, g), dict(initial_state=f32(1, 2, 64, 64).bfloat16()), "initial_state must be"),
        ((q, q, q, g), dict(cu_seqlens=[0, 4, 10], initial_state=pool[:2], state_out=pool[1:]), "overlap"),
        ((q.half(), q.half(), q.half(), g.half()), {}, "unsupported dtype"),
    ]:
        with pytest.raises(ValueError, match=text):
            api.gated_prefill(*args, **kw)


def test_backward_binding(stub):
    q, g = bf(10, 2, 64), bf(10, 2)
    with pytest.raises(Reached):
        api.gated_prefill_backward(q, q, q, g, q)
    with pytest.raises(Reached):
        api.gated_prefill_backward(q, q, q, None, q, cu_seqlens=[0, 3, 10], initial_state=f32(2, 2, 64, 64),
                                   d_state=f32(2, 2, 64, 64))
    for args, kw, text in [
        ((q, q, q, g, bf(9, 2, 64)), {}, "do must have shape"),
        ((q, q, q, g, f32(10, 2, 64)), {}, "do must be"),
        ((q, q, q, g, q), dict(d_state=f32(2, 2, 64, 64)), "d_state must have shape"),
        ((q, q, q, g, q), dict(initial_state=f32(1, 2, 64, 32)), "initial_state must have shape"),
    ]:
        with pytest.raises(ValueError, match=text):
            api.gated_prefill_backward(*args, **kw)


def test_decode_binding(stub):
    q, g, pool = bf(3, 2, 64), bf(3, 2), f32(5, 2, 64, 64)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(Reached):
        api.gated_decode_step(q, q, q, g, pool, slots=slots)
    with pytest.raises(Reached):
        api.gated_decode_step(q, q, q, None, f32(3, 2, 64, 64))
    for args, kw, text in [
        ((q, q, q, g, pool), {}, "without slots"),
        ((q, q, q, g, f32(5, 2, 64, 32)), dict(slots=slots), "state must be"),
        ((q, q, q, g, pool), dict(slots=slots.long()), "slots must be"),
        ((q, q, q, g, pool), dict(slots=slots[:2]), "slots must have shape"),
        ((q, q, q, bf(3, 3), pool), dict(slots=slots), "g must have shape"),
        ((q, q, q, g, pool), dict(slots=slots, out=q), "overlap"),
        ((bf(3, 2, 1, 64),) * 3 + (g, pool), {}, r"q must be \[B, H, D\]"),
    ]:
        with pytest.raises(ValueError, match=text):
            api.gated_decode_step(*args, **kw)


def test_host_tensors_are_refused():
    q = bf(8, 2, 64)
    for call in (lambda: api.gated_prefill(q, q, q, None), lambda: api.gated_prefill_backward(q, q, q, None, q),
                 lambda: api.gated_decode_step(q, q, q, None, f32(8, 2, 64, 64))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def _cu(cu):
    arr = np.ascontiguousarray(np.asarray(cu, np.int32))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(cu) - 1


BAD = [
    (dict(q=None), api.LA_ERR_INVALID_ARG), (dict(o=None), api.LA_ERR_INVALID_ARG),
    (dict(q=FAKE + 2), api.LA_ERR_INVALID_ARG), (dict(g=FAKE + 1), api.LA_ERR_INVALID_ARG),
    (dict(H=0), api.LA_ERR_INVALID_ARG), (dict(N=-1), api.LA_ERR_INVALID_ARG), (dict(B=0), api.LA_ERR_INVALID_ARG),
    (dict(D=96), api.LA_ERR_UNSUPPORTED), (dict(D=256), api.LA_ERR_UNSUPPORTED),
    (dict(flags=1 | 2), api.LA_ERR_INVALID_ARG), (dict(flags=1 | 4), api.LA_ERR_INVALID_ARG),
    (dict(st=FAKE + 8), api.LA_ERR_INVALID_ARG), (dict(ws=FAKE + 8), api.LA_ERR_INVALID_ARG),
    (dict(size=0, N=5000), api.LA_ERR_INVALID_ARG), (dict(ws=None, N=5000), api.LA_ERR_INVALID_ARG),
    (dict(cu=[0, 5, 3, 8]), api.LA_ERR_INVALID_ARG), (dict(cu=[1, 8]), api.LA_ERR_INVALID_ARG),
    (dict(cu=[0, 7]), api.LA_ERR_INVALID_ARG), (dict(cu=[0, 8], B=2), api.LA_ERR_INVALID_ARG),
    (dict(cu=list(range(1026)), N=1025), api.LA_ERR_UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 16), api.LA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_sequence_calls_reject(L, kw, code):
    a = dict(q=FAKE, o=FAKE, g=FAKE, B=1, H=2, N=8, D=128, flags=1, st=FAKE, ws=FAKE, size=1 << 60, cu=None)
    a.update(kw)
    keep, cu, n = (None, None, 0) if a["cu"] is None else _cu(a["cu"])
    shape = (a["B"], a["H"], a["N"], a["D"], cu, n, a["flags"])
    assert L.la_gated_prefill(a["q"], FAKE, FAKE, a["g"], a["o"], *shape, a["st"], a["st"], a["ws"], a["size"],
                              None) == code
    assert L.la_gated_prefill_backward(a["q"], FAKE, FAKE, a["g"], FAKE, a["o"], FAKE, FAKE, a["g"], *shape,
                                       a["st"], a["st"], a["st"], a["ws"], a["size"], None) == code


def test_backward_rejects_a_gate_gradient_without_gate(L):
    assert L.la_gated_prefill_backward(FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 2, 8, 128, None, 0, 1,
                                       None, None, None, FAKE, 1 << 60, None) == api.LA_ERR_INVALID_ARG


def test_workspace_sizes(L):
    n = ctypes.c_ulonglong()
    assert L.la_gated_workspace(1, 2, 8, 128, None, 0, 1, 0, None) == api.LA_ERR_INVALID_ARG
    assert L.la_gated_workspace(1, 2, 8, 96, None, 0, 1, 0, ctypes.byref(n)) == api.LA_ERR_UNSUPPORTED
    sizes = []
    for N in (0, 1, 100, 10000, 100000):
        for back in (0, 1):
            assert L.la_gated_workspace(1, 2, N, 128, None, 0, 0, back, ctypes.byref(n)) == api.LA_OK
            sizes.append(n.value)
    assert sizes[0] == 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), api.LA_ERR_INVALID_ARG), (dict(state=None), api.LA_ERR_INVALID_ARG),
    (dict(state=FAKE + 4), api.LA_ERR_INVALID_ARG), (dict(g=FAKE + 1), api.LA_ERR_INVALID_ARG),
    (dict(slots=FAKE + 2), api.LA_ERR_INVALID_ARG), (dict(B=-1), api.LA_ERR_INVALID_ARG),
    (dict(H=0), api.LA_ERR_INVALID_ARG), (dict(D=32), api.LA_ERR_UNSUPPORTED),
    (dict(slots=None, pool=1), api.LA_ERR_INVALID_ARG), (dict(flags=3), api.LA_ERR_INVALID_ARG),
    (dict(pool=-1), api.LA_ERR_INVALID_ARG), (dict(B=1 << 20, H=1 << 12), api.LA_ERR_UNSUPPORTED),
    (dict(B=65537, H=1, pool=65537), api.LA_ERR_UNSUPPORTED), (dict(B=0), api.LA_OK),
])
def test_decode_rejects(L, kw, code):
    a = dict(q=FAKE, g=FAKE, state=FAKE, B=2, H=2, D=128, slots=FAKE, pool=4, flags=1)
    a.update(kw)
    assert L.la_gated_decode_step(a["q"], FAKE, FAKE, a["g"], a["state"], FAKE, a["B"], a["H"], a["D"], a["slots"],
                                  a["pool"], a["flags"], None) == code
