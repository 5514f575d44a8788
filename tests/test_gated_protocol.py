"""What the gated kernels' barriers order, checked on the CPU: one property of the source, and
executable models of the three tensor-core kernels (``gated_protocol.py``) under random schedules,
which have to be clean for every shape of call and to catch each planted mistake.
"""
import os
import re

import pytest

from gated_protocol import BackwardModel, PrefillModel, StateModel
from pair_protocol import ProtocolError

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_04_b200", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_tile_reads_are_fenced_before_tma_refills_the_place():
    """The gradient kernel's scaling group reads rows of the q and k tiles by ordinary loads; its
    arrival on `scaled` leads, through the products behind it, to the TMA loads that take those
    tiles' places.  Ordinary reads and TMA writes belong to different proxies, which an mbarrier
    does not order: the proxy fence has to stand between the last read and the arrival."""
    text = _source("gated_backward_tc.cuh")
    reads = [m.end() for m in re.finditer(r"scale\(C::TM_D[QK], ", text)]
    arrival = text.index("mbar_arrive(&m->scaled)")
    assert len(reads) == 2 and max(reads) < arrival
    assert "fence_proxy_async_smem();" in text[max(reads):arrival]


def _first_violation(make, seeds):
    for seed in range(seeds):
        try:
            make().run(seed)
        except ProtocolError as e:
            return str(e)
    return None


@pytest.mark.parametrize("tails", [[False], [True], [False] * 4, [True, False, True], [False, True, True, False, False]])
@pytest.mark.parametrize("stream", [True, False], ids=["d128", "d64"])
@pytest.mark.parametrize("have_s", [True, False], ids=["s", "no-s"])
@pytest.mark.parametrize("have_ds", [True, False], ids=["ds", "no-ds"])
def test_gradients(tails, stream, have_s, have_ds):
    assert _first_violation(lambda: BackwardModel(tails, stream, have_s, have_ds), 12) is None


@pytest.mark.parametrize("nb", [0, 1, 2, 3, 4, 7])
@pytest.mark.parametrize("tail", [False, True], ids=["full", "tail"])
@pytest.mark.parametrize("slots,through,snap", [(3, False, True), (3, False, False), (2, True, True), (3, True, True),
                                                (2, False, True)])
def test_states(nb, tail, slots, through, snap):
    assert _first_violation(lambda: StateModel(nb, tail and nb > 0, slots, through, snap), 12) is None


@pytest.mark.parametrize("nb", [0, 1, 2, 3, 4, 7])
@pytest.mark.parametrize("tail", [False, True], ids=["full", "tail"])
def test_prefill(nb, tail):
    assert _first_violation(lambda: PrefillModel(nb, tail and nb > 0), 20) is None


# mistake -> words of which the violations found must name one
GRADIENTS = {
    "low_no_wait": ("low", ),                  # the next columns over those a product still reads
    "vo_early": ("v", "do"),                   # v, do loaded once k dS is done, before P^T do
    "qs_early": ("q", "s"),                    # q, S loaded once dq is done, before dP^T q
    "no_tail_wait": ("zeroed", "fence"),       # products of rows behind the sequence
    "first_full_early": ("v0", "v1", "tdk"),   # P over v before the last columns of dS's second part
    "no_scaled_wait": ("tdq", "tdk"),          # second terms added before the first were scaled
    "no_dg_wait": ("rowcol", "lands in phase"),  # sums overwritten before dg has read them
    "no_fence_p": ("fence",), "no_fence_b": ("fence",), "no_fence_tail": ("fence",),
    "no_low_wait": ("tdq",),                   # dq's first term scaled before its second part is there
}
STATES = {
    "slice_no_wait": ("slice",), "no_acc_free": ("acc",), "gates_no_wait": ("sums", "lands in phase"),
    "no_store_wait": ("out",), "no_parts_wait": ("parts", "slice"),
    "no_fence_other": ("fence",), "no_fence_snap": ("fence",), "no_fence_parts": ("fence",),
}
PREFILL = {
    "k_no_wait": ("k0", "k1"), "q_no_wait": ("q0", "q1"), "v_no_wait": ("v0", "v1"), "no_o_free": ("scores",),
    "no_o_free2": ("qS", "Pv"), "no_tail_wait": ("zeroed", "fence"), "no_kv_free": ("kv",), "no_qs_wait": ("snap",),
    "no_split_wait": ("v0", "v1", "lands in phase"), "no_read_wait": ("v0", "v1"), "no_v_free": ("v'",),
    "no_fence_snap": ("fence",), "no_fence_o": ("fence",), "no_fence_v": ("fence",), "no_fence_tail": ("fence",),
}


def _caught(make, words):
    said = []
    for seed in range(200):
        try:
            make().run(seed)
        except ProtocolError as e:
            said.append(str(e))
    assert said, "no schedule shows it"
    assert any(w in e for e in said for w in words), said[:3]


@pytest.mark.parametrize("mutant", GRADIENTS)
def test_gradients_mutants(mutant):
    _caught(lambda: BackwardModel([False, False, True, False], mutations=(mutant,)), GRADIENTS[mutant])


@pytest.mark.parametrize("mutant", STATES)
def test_states_mutants(mutant):
    _caught(lambda: StateModel(6, True, 2, True, mutations=(mutant,)), STATES[mutant])


@pytest.mark.parametrize("mutant", PREFILL)
def test_prefill_mutants(mutant):
    _caught(lambda: PrefillModel(5, True, mutations=(mutant,)), PREFILL[mutant])
