"""What may not cross the C boundary, and sizes at its edge (CPU)."""
import ctypes
import subprocess

import numpy as np
import pytest

from long_context_04_b200 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_nothing_can_throw_behind_a_c_entry():
    """An exception that leaves a C entry ends the process.  The library allocates nothing that
    throws and throws nothing itself: it imports no such function."""
    build.build()
    names = subprocess.run(["nm", "-D", "--undefined-only", build.LIB], capture_output=True, text=True,
                           check=True).stdout.split()
    bad = [n for n in names if n.startswith(("_ZSt", "_Znw", "_Zna", "__cxa_throw", "__cxa_rethrow"))]
    assert not bad, bad


def _order(L, lengths, flags=1):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    n = ctypes.c_ulonglong()
    rc = L.la_gated_workspace(1, 2, int(cu[-1]), 64, cu.ctypes.data, len(lengths), flags, 1, ctypes.byref(n))
    return rc, n.value


def test_a_plan_does_not_depend_on_the_order_of_the_sequences(L):
    gen = np.random.default_rng(3)
    lengths = gen.integers(0, 900, 1024)
    want = _order(L, lengths)
    assert want[0] == api.LA_OK and want[1] > 0
    for _ in range(3):
        gen.shuffle(lengths)
        assert _order(L, lengths) == want
    assert _order(L, np.sort(lengths)) == want and _order(L, np.full(1024, 300))[0] == api.LA_OK


@pytest.mark.parametrize("flags", [0, 1], ids=["fp32", "bf16"])
@pytest.mark.parametrize("backward", [0, 1], ids=["prefill", "backward"])
def test_lengths_next_to_2_31_are_refused(L, flags, backward):
    """2^31 - 1 tokens have more snapshot rows than a coordinate holds: refused, and not counted
    as no blocks because the rounded-up length left 32 bits."""
    n = ctypes.c_ulonglong(7)
    for N in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 127):
        assert L.la_gated_workspace(1, 1, N, 64, None, 0, flags, backward, ctypes.byref(n)) == api.LA_ERR_UNSUPPORTED
        cu = np.asarray([0, N], np.int32)
        assert L.la_gated_workspace(1, 1, N, 64, cu.ctypes.data, 1, flags, backward,
                                    ctypes.byref(n)) == api.LA_ERR_UNSUPPORTED
    assert n.value == 7
