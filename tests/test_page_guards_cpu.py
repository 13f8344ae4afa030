"""Chunk attention and page operators without a GPU: what their sources must not
hold, the guard of the join of pieces, and refusals."""
import ctypes
import glob
import os
import re
import subprocess

import torch

from paged_kv_cache_loc_gb300 import _lib, build
from test_abi import O, Q, ROOT, fake_cache

CSRC = os.path.join(ROOT, "paged_kv_cache_loc_gb300", "csrc")


def build_and_load():
    build.build()
    return _lib.load()


def test_no_copy_goes_to_several_ctas():
    """A pool may lie in any memory that the GPU can address, and every rank of a
    run on several GPUs loads this library: a TMA load with cluster multicast
    must not meet another GPU's memory, so there is none."""
    sources = [f for ext in ("*.cu", "*.cuh", "*.h", "*.cpp") for f in glob.glob(os.path.join(CSRC, ext))]
    assert len(sources) > 10
    assert [f for f in sources if "multicast" in open(f).read()] == []


def test_join_takes_no_unwritten_pair(tmp_path):
    """The words that name an item's pieces lie in the caller's workspace, and a
    wait that gives up leaves them unwritten.  Whatever stands there, the pieces
    are ones that the workspace has room for: CTAs 0 .. parts - 1."""
    prog = tmp_path / "pieces.cu"
    prog.write_text(r'''
#include <stdio.h>
#include "pkv_chunk_join.cuh"
int main() {
  int first, last, parts;
  while (scanf("%d %d %d", &first, &last, &parts) == 3) printf("%d\n", pkv::item_pieces(first, last, parts));
  return 0;
}''')
    exe = tmp_path / "pieces"
    subprocess.check_call([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(prog), "-o", str(exe)])
    top = 2**31 - 1
    words = [-top - 1, -top, -1, 0, 1, 2, 150, 151, 152, 153, 0x3F800000, 0x7FC00000, top - 1, top]    # 1.0 and NaN among them
    asked = [(a, b, n) for a in words for b in words for n in (1, 2, 152)]
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % x for x in asked), capture_output=True, text=True, check=True).stdout
    got = [int(x) for x in out.split()]
    assert len(got) == len(asked)
    for (a, b, n), pieces in zip(asked, got):
        assert pieces == (b - a + 1 if 0 <= a < b < n else 0), (a, b, n)


def test_chunk_refuses_contexts_of_more_positions_than_its_sums_hold():
    """2^30 positions at most: pieces' ends are summed in 32 bits.  (A table may
    name a page many times, so the pool's size does not bound a context.)"""
    lib = build_and_load()

    def call(max_len, dtype, max_q):
        c = fake_cache(qo_indptr=0x9000, max_len=max_len, dtype=dtype, n_kv_heads=1)
        return lib.pkv_paged_chunk(ctypes.byref(c), 0, ctypes.c_void_p(0x1000), 1 << 24, 128, Q, O, 4, 1, max_q, 1, 0.1, None, None)

    for dtype in (_lib.PKV_F32, _lib.PKV_BF16):
        for max_q in (1, 4, 500):
            for max_len in (2**30 + 1, 2**31 - 128, 2**31 - 1):
                assert call(max_len, dtype, max_q) == _lib.PKV_ERR_ARG
                c = fake_cache(qo_indptr=0x9000, max_len=max_len, dtype=dtype, n_kv_heads=1)
                assert lib.pkv_chunk_workspace_bytes(ctypes.byref(c), 4, 1, max_q) == 0
            if not torch.cuda.is_available():     # not refused: it asks for the device
                assert call(2**30, dtype, max_q) == _lib.PKV_ERR_CUDA


def test_every_code_of_a_wait_is_documented():
    """The codes that kernels record when a wait gives up, and the list at
    pkv_last_device_error: the same numbers, none left out, none that is gone."""
    recorded = set()
    for f in glob.glob(os.path.join(CSRC, "*.cu")):
        recorded |= {int(x) for x in re.findall(r"(?:give_up\(|record_error\(p\.err, )-(\d{4,5})[,)]", open(f).read())}
    text = open(os.path.join(ROOT, "include", "pkv.h")).read()
    text = text[text.index("one of these codes"):text.index("int pkv_last_device_error")]
    listed = set()
    for a, b in re.findall(r"-(\d{4})(?!\d)(?: \.\. -(\d{4})(?!\d))?", text):
        listed |= set(range(int(a), int(b or a) + 1))
    assert recorded and recorded <= listed, recorded - listed
    assert {x for x in listed if x >= 5000} == {x for x in recorded if x >= 5000}
