"""What the gated kernels' barriers order, checked on the CPU."""
import os
import re

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
