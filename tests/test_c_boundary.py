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
