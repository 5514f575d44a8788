"""Sequence boundaries that a host array holds in other types than int32 (CPU)."""
import numpy as np
import pytest
import torch

from long_context_04_b200 import api


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def stub(monkeypatch):
    monkeypatch.setattr(api, "_on_gpu", lambda t: True)

    def reached():
        raise Reached()
    monkeypatch.setattr(api, "lib", reached)


def calls():
    q, g = torch.zeros(10, 2, 64, dtype=torch.bfloat16), torch.zeros(10, 2, dtype=torch.bfloat16)
    return [lambda cu: api.prefill(q, q, q, cu_seqlens=cu), lambda cu: api.chunk_state(q, q, cu_seqlens=cu),
            lambda cu: api.gated_prefill(q, q, q, g, cu_seqlens=cu),
            lambda cu: api.gated_prefill_backward(q, q, q, g, q, cu_seqlens=cu)]


@pytest.mark.parametrize("call", calls(), ids=["prefill", "chunk_state", "gated_prefill", "gated_prefill_backward"])
def test_boundaries(call):
    for good in ([0, 4, 10], (0, 4, 10), np.asarray([0, 4, 10]), np.asarray([0, 4, 10], np.int32),
                 np.asarray([0, 4, 10], np.uint64), np.asarray([0.0, 4.0, 10.0]), torch.tensor([0, 4, 10]),
                 torch.tensor([0, 4, 10], dtype=torch.int32)):
        with pytest.raises(Reached):
            call(good)
    # 2^32 + 4 is 4 in 32 bits, 4.7 is 4 as a whole number
    for bad in (np.asarray([0, 2 ** 32 + 4, 10]), torch.tensor([0, 2 ** 32 + 4, 10]), [0, 2 ** 32 + 4, 10],
                np.asarray([0, 2 ** 63 + 4, 10], np.uint64), [0, 4.7, 10], np.asarray([0, 4.7, 10]),
                np.asarray([0, np.nan, 10]), [[0], [4], [10]], np.asarray([[0, 10]])):
        with pytest.raises(ValueError, match="cu_seqlens"):
            call(bad)
