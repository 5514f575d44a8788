"""A call on another stream while the current stream still uses freed memory of its results' size."""
import pytest
import torch

from gated_cases import inputs
from long_context_04_b200 import api

pytestmark = pytest.mark.gpu

T, H, D = 300, 2, 128


def _calls():
    x = inputs([0, T], H, D, torch.bfloat16, 61, "cuda", grad=True, states=True)
    q, k, v, g = (x[n] for n in "qkvg")
    tok = [t[:1].contiguous() for t in (q, k, v, g)]
    gathered = torch.stack([x["initial"], x["d_state"]])
    states = [x["initial"].clone() for _ in range(3)]   # one for each call, made before the sleep
    return {
        "prefill": lambda s: api.prefill(q, k, v, return_state=True, stream=s),
        "decode_step": lambda s: (api.decode_step(*tok[:3], states.pop(), stream=s),),
        "chunk_state": lambda s: (api.chunk_state(k, v, stream=s),),
        "state_prefix": lambda s: (api.state_prefix(gathered, 2, stream=s),),
        "gated_prefill": lambda s: api.gated_prefill(q, k, v, g, return_state=True, stream=s),
        "gated_prefill_backward": lambda s: api.gated_prefill_backward(
            q, k, v, g, x["do"], initial_state=x["initial"], d_state=x["d_state"], stream=s),
        "gated_decode_step": lambda s: (api.gated_decode_step(*tok, states.pop(), stream=s),),
    }


@pytest.mark.parametrize("name", ["prefill", "decode_step", "chunk_state", "state_prefix", "gated_prefill",
                                  "gated_prefill_backward", "gated_decode_step"])
def test_freed_memory_still_in_use(name):
    """The current stream sleeps, then fills tensors that are freed before it gets there.  The
    call's results, on another stream, have to come from elsewhere."""
    call = _calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    call(side)  # the side stream's pool has its blocks
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    held = [torch.empty_like(t) for t in want for _ in range(2)]
    for t in held:
        t.fill_(7.0)
    del held, t
    got = call(side)
    side.synchronize()
    late = [t.clone() for t in got]     # on the current stream: behind the fills
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    for a, b in zip(want, late):
        assert torch.equal(a, b)


def test_arguments_freed_at_once():
    """Arguments that are freed when the call returns, while its stream has not begun."""
    x = inputs([0, T], H, D, torch.bfloat16, 62, "cuda")
    want = api.gated_prefill(*(x[n] for n in "qkvg")).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    side_args = [x[n].clone() for n in "qkvg"]
    torch.cuda.current_stream().synchronize()   # the copies are made; the call's stream still sleeps
    got = api.gated_prefill(*side_args, stream=side)
    del side_args
    for n in "qkvg":
        torch.full_like(x[n], 7.0)              # would take the freed blocks
    torch.cuda.synchronize()
    assert api.device_status() == api.LA_OK
    assert torch.equal(got, want)


def test_capture_with_a_forked_stream():
    """A capture whose call runs on a second stream, forked from the captured one and joined."""
    x = inputs([0, T], H, D, torch.bfloat16, 63, "cuda", grad=True, states=True)

    def call(s=None):
        a = api.gated_prefill(*(x[n] for n in "qkvg"), initial_state=x["initial"], return_state=True, stream=s)
        return a + api.gated_prefill_backward(*(x[n] for n in "qkvg"), x["do"], initial_state=x["initial"],
                                              d_state=x["d_state"], stream=s)

    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(side)
        here.wait_stream(side)
    for seed in (64, 65):
        for n, t in inputs([0, T], H, D, torch.bfloat16, seed, "cuda", grad=True, states=True).items():
            x[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert api.device_status() == api.LA_OK
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


def test_captured_decode_reads_the_slots_of_its_replay():
    x = inputs([0, 4], H, D, torch.bfloat16, 66, "cuda")
    gen = torch.Generator().manual_seed(9)
    start = torch.randn(6, H, D, D, generator=gen).cuda()
    pool, slots = start.clone(), torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    api.gated_decode_step(*(x[n] for n in "qkvg"), pool, slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = api.gated_decode_step(*(x[n] for n in "qkvg"), pool, slots=slots)
    for at in ([5, 3, 0, 1], [2, -1, 4, 5]):
        pool.copy_(start)
        slots.copy_(torch.tensor(at, dtype=torch.int32))
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert api.device_status() == api.LA_OK
        rows = [b for b, s in enumerate(at) if s >= 0]
        own = start[[at[b] for b in rows]].contiguous()
        y = api.gated_decode_step(*(x[n][rows].contiguous() for n in "qkvg"), own)
        torch.cuda.synchronize()
        assert torch.equal(o[rows], y) and torch.equal(pool[[at[b] for b in rows]], own)
        rest = [s for s in range(6) if s not in at]
        assert torch.equal(pool[rest], start[rest])
        assert all(bool((o[b] == 7).all()) for b, s in enumerate(at) if s < 0)
