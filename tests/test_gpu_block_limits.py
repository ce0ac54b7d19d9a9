"""GPU tests of the pre-norm block's operators where their waits and numbers end."""
import time

import pytest
import torch

from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import MoEConfig

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TIMEOUT, SITE = 1, 900


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d,row", [(1, 1088, 0), (40, 2048, 39), (3000, 2560, 7), (1500, 4096, 1300), (700, 7168, 500),
                                     (40, 8256, 3), (600, 12288, 410), (300, 32768, 120)])
def test_layernorm_wait_that_runs_out(n, d, row, kind):
    """A row that never arrives: its wait ends after 50 us, the row and the later ones of the same blocks
    are not a number, every other row is what it is without, and the next call is whole again."""
    desc = api.make_desc(MoEConfig("late", n, d, 64, 8, 2))
    ws = torch.empty(api.moe_workspace_size(desc)[1], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    g = torch.Generator().manual_seed(n + d)
    x = torch.randn(n, d, generator=g).to(kind).cuda()
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma = torch.randn(d, generator=g).cuda()

    def forward(late):
        y = torch.zeros(n, d, dtype=BF16, device="cuda")
        mean, rstd = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        if late:
            api.moe_selftest_layernorm_timeout(desc, x, gamma, mean, rstd, row, 50_000, ws, y=y)
        else:
            api.moe_layernorm(desc, x, gamma, None, y, mean, rstd)
        torch.cuda.synchronize()
        return y, mean, rstd

    def backward(late, mean, rstd):
        dx, dg, db = torch.zeros_like(x), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
        if late:
            api.moe_selftest_layernorm_timeout(desc, x, gamma, mean, rstd, row, 50_000, ws, dy=dy, dx=dx, dgamma=dg,
                                               dbeta=db)
        else:
            api.moe_layernorm_backward(desc, dy, x, gamma, mean, rstd, None, dx, dg, db, ws)
        torch.cuda.synchronize()
        return dx, dg, db

    def lost(t):                                   # rows that are not a number, which is all of the row or none of it
        nan = torch.isnan(t)
        assert torch.equal(nan.all(1), nan.any(1))
        return nan.any(1)

    clean = forward(False)
    t0 = time.perf_counter()
    y, mean, rstd = forward(True)
    assert time.perf_counter() - t0 < 1.0          # not the ordinary limit of two seconds
    bad = lost(y)
    assert bad[row] and not bad[:row].all() or row == 0
    assert torch.equal(torch.isnan(mean), bad) and torch.equal(torch.isnan(rstd), bad)
    for a, b in zip((y, mean, rstd), clean):
        assert torch.equal(a[~bad], b[~bad])
    if n <= 40:                                    # a block a row: no other is lost
        assert int(bad.sum()) == 1
    assert api.moe_get_device_status(ws) == (0, 0)

    gclean = backward(False, *clean[1:])
    dx, dg, db = backward(True, *clean[1:])
    bad = lost(dx)
    assert bad[row] and torch.equal(dx[~bad], gclean[0][~bad])
    if n <= 40:
        assert int(bad.sum()) == 1
    assert torch.isnan(dg).all() and torch.isnan(db).all()
    assert api.moe_get_device_status(ws) == (TIMEOUT, SITE)
    api.moe_workspace_init(ws)
    for a, b in zip(forward(False) + backward(False, *clean[1:]), clean + gclean):
        assert torch.equal(a, b)
    assert api.moe_get_device_status(ws) == (0, 0)
