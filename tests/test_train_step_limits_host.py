"""Limits of the training step's operators that need no GPU: index arithmetic at large sizes, workspace sizes."""
import subprocess

import pytest
import torch

from ragged_grouped_gemm_gb300 import api, build
from ragged_grouped_gemm_gb300.inputs import MoEConfig

RUNS = r"""
#include <cstdio>
#include <initializer_list>
#include "row_runs.h"
// Every k-block belongs to one run, in order, and no run is empty or longer than a run and a k-block.
int main() {
  const int rows[] = {0, 1, 64, 1791, 1792, 1793, 3584, 3585, 8192, 1000003, 15700000, 16777216, 22300000, 33554433,
                      1 << 27, (1 << 30) + 1, 2147483647 - 256};
  for (int r : rows)
    for (int kb : {64, 128}) {
      const int runs = moe::row_runs(r), n = (r + kb - 1) / kb;
      bool ok = runs >= 1 && (runs == 1) == (r <= moe::kRowChunk) && moe::run_begin(0, runs, n) == 0 &&
                moe::run_begin(runs, runs, n) == n;
      for (int i = 0; i < runs; ++i) {
        const int len = moe::run_begin(i + 1, runs, n) - moe::run_begin(i, runs, n);
        ok = ok && (len > 0 || n == 0) && len <= moe::kRowChunk / kb + 1;
      }
      std::printf("%d %d %d\n", r, kb, ok);
    }
}
"""


def test_runs_of_rows_cover_a_group(tmp_path):
    src, exe = tmp_path / "runs.cpp", tmp_path / "runs"
    src.write_text(RUNS)
    subprocess.run(["g++", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    assert len(lines) == 34 and all(line.endswith(" 1") for line in lines), lines


@pytest.mark.parametrize("n,d,f,e,k,most", [
    (16384, 4096, 512, 512, 1, 317070336), (4096, 1024, 64, 1024, 1, 82879488), (1, 4096, 14336, 8, 2, 1661952),
    (2, 65536, 64, 1001, 1, 264295680)])
def test_workspaces_hold_the_layer_alone(n, d, f, e, k, most):
    """The dense router gradient works in what the layer has: sizes as they were before it came."""
    build.build()
    assert api.moe_workspace_size(api.make_desc(MoEConfig("case", n, d, f, e, k)))[1] <= most


@pytest.mark.parametrize("checkpoint", [False, True])
def test_layer_needs_a_forward(monkeypatch, checkpoint):
    """Buffers that no forward has written hold any index: nothing is enqueued on them."""
    layer = object.__new__(api.MoELayer)
    vars(layer).update(train=True, cap=False, checkpoint=checkpoint, x=None, kept=False, balance=None, grads={})
    for name in ("moe_backward", "moe_backward_ckpt", "moe_balance_loss"):
        monkeypatch.setattr(api, name, lambda *a, **k: pytest.fail("enqueued"))
    with pytest.raises(ValueError, match="needs the forward"):
        layer.backward(None)
    with pytest.raises(ValueError, match="needs the forward"):
        layer.balance_loss(torch.zeros(2, dtype=torch.int32), 0.01)
    layer.train = False
    with pytest.raises(ValueError, match="train=False"):
        layer.backward(None)
