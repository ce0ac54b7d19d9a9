"""Limits of the block's entry points and kernels that hold on the CPU."""
import glob
import os
import re

from ragged_grouped_gemm_gb300 import build


def _sources():
    return {os.path.basename(p): open(p).read() for p in glob.glob(os.path.join(build.CSRC, "*.cu*"))}


def test_every_aligned_cluster_barrier_converges_its_warp_first():
    """`barrier.cluster.*.aligned` is undefined for a warp whose lanes do not arrive together, and a
    branch of some lanes may stand right before any call: the convergence belongs to the barrier's
    own wrapper, and no other code issues it."""
    found = []
    for name, text in _sources().items():
        for m in re.finditer(r"barrier\.cluster\.arrive", text):
            body = text[text.rfind("{", 0, m.start()):m.start()]
            found.append(name)
            assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"$", body), (name, body)
    assert found == ["sm100_ptx.cuh"]
