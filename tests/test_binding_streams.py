"""Calls on a stream that is not the current one: whose memory the binding hands to the kernels.

The caching allocator gives a freed block out again at once on the stream it was allocated on,
because work there runs in order.  A kernel on another stream is not in that order: what a call
allocates has to come from the pool of the stream it runs on, be kept for the current stream too
(the caller reads it there), and what the caller passes has to be kept for the call's stream.
Here CPU tensors, a stub library and recorded streams stand in for the GPU.
"""
import contextlib

import pytest
import torch

from long_context_04_b200 import api


class Fake:
    def __init__(self, name):
        self.name, self.cuda_stream = name, hash(name) & 0xffff
        self.device = torch.device("cpu")

    def __eq__(self, other):
        return self.name == other.name


class Library:
    """Every entry point returns LA_OK; the workspace call names one byte."""

    def __getattr__(self, name):
        def call(*args):
            if name == "la_gated_workspace":
                args[-1]._obj.value = 1
            return api.LA_OK
        return call


@pytest.fixture
def world(monkeypatch):
    """current: stack of current streams; born: storage -> stream; kept: storage -> streams."""
    w = dict(current=[Fake("here")], born={}, kept={})
    monkeypatch.setattr(api, "_on_gpu", lambda t: True)
    monkeypatch.setattr(api, "lib", Library)

    @contextlib.contextmanager
    def stream(s):
        w["current"].append(s)
        try:
            yield
        finally:
            w["current"].pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w["current"][-1])
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: w["kept"].setdefault(t.data_ptr(), set()).add(s.name))
    for name in ("empty", "empty_like"):
        def made(*args, _make=getattr(torch, name), **kw):
            t = _make(*args, **kw)
            w["born"][t.data_ptr()] = w["current"][-1].name
            w.setdefault("all", []).append(t)   # kept alive: addresses stay distinct
            return t
        monkeypatch.setattr(torch, name, made)
    return w


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def calls():
    q, g, st = bf(10, 2, 64), bf(10, 2), f32(1, 2, 64, 64)
    a = [bf(10, 2, 64) for _ in range(4)]
    d, pool, slots = [bf(3, 2, 64) for _ in range(3)], f32(5, 2, 64, 64), torch.zeros(3, dtype=torch.int32)
    own, gd, gathered = f32(3, 2, 64, 64), bf(3, 2), f32(3, 1, 2, 64, 64)
    return {
        "prefill": (a[:3] + [st], lambda s: api.prefill(*a[:3], return_state=True, initial_state=st, stream=s)),
        "decode_step": (d + [own], lambda s: api.decode_step(*d, own, stream=s)),
        "state_out": ([own, pool, slots], lambda s: api.state_out(own, pool, slots, stream=s)),
        "chunk_state": (a[:2], lambda s: api.chunk_state(*a[:2], stream=s)),
        "state_prefix": ([gathered], lambda s: api.state_prefix(gathered, 1, stream=s)),
        "gated_prefill": (a[:3] + [g, st], lambda s: api.gated_prefill(*a[:3], g, return_state=True,
                                                                       initial_state=st, stream=s)),
        "gated_prefill_backward": (a + [g, st], lambda s: api.gated_prefill_backward(*a[:3], g, a[3], initial_state=st,
                                                                                     d_state=st, stream=s)),
        "gated_decode_step": (d + [gd, pool, slots], lambda s: api.gated_decode_step(*d, gd, pool, slots=slots,
                                                                                     stream=s)),
        "given outputs": (a[:3] + [a[3], st], lambda s: api.gated_prefill(*a[:3], g, out=a[3], state_out=st, stream=s)),
    }


@pytest.mark.parametrize("name", calls().keys())
def test_memory_of_a_call_on_another_stream(world, name):
    given, call = calls()[name]
    got = call(Fake("side"))
    for t in given:
        assert "side" in world["kept"].get(t.data_ptr(), ()), "an argument is not kept for the call's stream"
    for t in got if isinstance(got, tuple) else (got,):
        if any(t is x for x in given):
            continue
        assert world["born"][t.data_ptr()] == "side", "a result comes from another stream's pool"
        assert "here" in world["kept"].get(t.data_ptr(), ()), "a result is not kept for the current stream"


@pytest.mark.parametrize("name", calls().keys())
@pytest.mark.parametrize("stream", [None, Fake("here")], ids=["default", "current"])
def test_memory_of_a_call_on_the_current_stream(world, name, stream):
    calls()[name][1](stream)
    assert set(world["born"].values()) <= {"here"} and not world["kept"]
