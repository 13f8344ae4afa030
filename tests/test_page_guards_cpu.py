"""Chunk attention and page operators without a GPU: what their sources must not
hold, the guard of the join of pieces, and refusals."""
import glob
import os

from test_abi import ROOT

CSRC = os.path.join(ROOT, "paged_kv_cache_loc_gb300", "csrc")


def test_no_copy_goes_to_several_ctas():
    """A pool may lie in any memory that the GPU can address, and every rank of a
    run on several GPUs loads this library: a TMA load with cluster multicast
    must not meet another GPU's memory, so there is none."""
    sources = [f for ext in ("*.cu", "*.cuh", "*.h", "*.cpp") for f in glob.glob(os.path.join(CSRC, ext))]
    assert len(sources) > 10
    assert [f for f in sources if "multicast" in open(f).read()] == []
