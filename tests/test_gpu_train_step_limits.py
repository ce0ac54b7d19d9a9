"""GPU limits of the training step's operators: logits far from zero, workspaces of the least size, long groups, and
how exact the short chains of sums are, against 64-bit numpy, with bounds that count the roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import np32
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig, make_dy, make_layer

pytestmark = pytest.mark.gpu
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
U = 2.0 ** -24


def _balance(lg, idx, off, gate, coef=0.01, z=0.001, up=None):
    n, e = lg.shape
    desc = api.make_desc(MoEConfig("case", n, 64, 64, e, idx.shape[1], gate=gate))
    ws = torch.empty(api.moe_workspace_size(desc)[0], dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    counts = torch.full((len(off) - 1, e), -7, dtype=I32, device="cuda")
    loss, dl = torch.full((2,), 9.0, device="cuda"), torch.full((n, e), 5.0, device="cuda")
    api.moe_balance_loss(desc, lg, idx, torch.tensor(off, dtype=I32, device="cuda"), counts, loss, dl, ws, coef, z,
                         None if up is None else torch.tensor([up], device="cuda"))
    return counts, loss, dl


def _check_rows(lg, idx, gate, got, coef, z, up=1.0):
    """One sequence of all rows.  An exponential of l - m carries the rounding of the difference (|l - m| U) and two ulps
    of its own, a sigmoid two such and its quotient, a sum E / 32 + 5 roundings: a probability is off by
    r = 2 (E / 32 + 16 + 2 max|l - m|) U of itself, inner by as much, f - inner by r of (f + inner), and the products add
    eight roundings.  lse is off by r + |lse| U.  Every factor is a normal number, so this holds for each number by
    itself; what is below 2^-126 in the end is off by a few 2^-149."""
    lg64 = lg.cpu().double().numpy()
    n, e = lg64.shape
    rc, rl, rg = O.balance_loss(lg64, idx.cpu().numpy(), [0, n], gate, coef, z)
    np.testing.assert_array_equal(got[0].cpu().numpy(), rc)
    f = rc[0] / n
    low = np.where(np.isneginf(lg64), np.inf, lg64)
    m = lg64.max(axis=1, keepdims=True)
    live = np.isfinite(m[:, 0])
    m0 = np.where(np.isfinite(m), m, 0.0)
    span = np.where(live, (m0 - np.where(np.isfinite(low), low, m0)).max(axis=1), 0.0)
    r = 2 * (e / 32 + 16 + 2 * np.minimum(span, 200.0))[:, None] * U        # beyond 200 a term is zero on both sides
    p = np.exp(lg64 - m0)
    lse = np.where(live, m0[:, 0] + np.log(np.where(live, p.sum(1), 1.0)), 0.0)[:, None]
    p = p / np.where(live, p.sum(1), 1.0)[:, None]
    q, w = O.train_step.gate_rows(lg64, gate)
    inner = (q @ f)[:, None]
    assert abs(got[1][0].item() - rl[0]) <= (r.max() + U) * rl[0]
    big = np.abs(lse).max()
    assert abs(got[1][1].item() - rl[1]) <= 2 * z * big * (r.max() + big * U) + U * rl[1]
    tol = coef * e / n * w * (f + inner) * (2 * r + 8 * U)
    tol = tol + 2 * z / n * p * (np.abs(lse) * (2 * r + 8 * U) + r + np.abs(lse) * U)
    assert (np.abs(np32(got[2]).astype(np.float64) - up * rg) <= up * tol + 1e-43).all()


def _rows(n, e, k, level, seed):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(n, e, generator=g) * 1.3 + torch.tensor(level)[torch.arange(n) % len(level)][:, None]
    return lg.cuda(), lg.topk(k, dim=1).indices.to(I32).cuda()


SIZES = [(60, 48, 4), (200, 8, 2), (700, 60, 6), (900, 256, 8), (300, 1021, 3)]   # the first two: one cluster


@pytest.mark.parametrize("n,e,k", SIZES)
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_balance_of_logits_far_below_zero(gate, n, e, k):
    """Where every sigmoid of a row is below the smallest number, their ratios still are the gate's distribution."""
    lg, idx = _rows(n, e, k, [-29.0, -60.0, -85.0, -90.0, -95.0, -100.0, -103.0, -106.0, -150.0, -1000.0, 0.0, -20.0], n)
    lg[5, 1:], lg[6, :], lg[7, 1:e // 2] = -float("inf"), -float("inf"), -float("inf")
    for coef, z in ((0.01, 0.0), (0.01, 0.001)):
        _check_rows(lg, idx, gate, _balance(lg, idx, [0, n], gate, coef, z), coef, z)
    lg[8] = torch.finfo(F32).min                                   # log sum beyond 1e19: no z-loss here
    lg[9, 1:] = torch.finfo(F32).min
    _check_rows(lg, idx, gate, _balance(lg, idx, [0, n], gate, 0.01, 0.0), 0.01, 0.0)


@pytest.mark.parametrize("n,e,k", SIZES)
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("z", [0.0, 0.001])
def test_balance_of_a_logit_that_is_no_number(gate, n, e, k, value, z):
    """Its row and the losses are NaN (the z-loss where there is one), every other row is what it was."""
    lg, idx = _rows(n, e, k, [0.0, 2.0], n)
    lg[3, :e // 2] = -float("inf")
    clean = _balance(lg, idx, [0, n - 2], gate, z=z)
    lg[3, e - 1] = lg[n - 1, 0] = value                                        # the second in no sequence
    got = _balance(lg, idx, [0, n - 2], gate, z=z)
    assert torch.isnan(got[2][3]).all() and torch.isnan(got[1][0])
    assert torch.isnan(got[1][1]) if z else got[1][1] == 0
    rest = [i for i in range(n) if i != 3]
    assert torch.equal(got[2][rest], clean[2][rest]) and torch.equal(got[0], clean[0])


@pytest.mark.parametrize("n,e,k", SIZES + [(20000, 8, 2)])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("up", [1.0, 1024.0])
def test_balance_of_logits_far_above_zero(gate, n, e, k, up):
    """A small factor of a row with a large sum of exponentials keeps its bits."""
    lg, idx = _rows(n, e, k, [20.0, 30.0, 34.0, 36.0, 45.0, 66.0, 68.0, 72.0, 74.0, 76.0, 85.0, 90.0, 0.0, 1000.0], n)
    for coef, z in ((1e-5, 0.0), (1e-5, 1e-5), (0.0, 1e-7), (1e-8, 0.0)):
        _check_rows(lg, idx, gate, _balance(lg, idx, [0, n], gate, coef, z, up), coef, z, up)


def test_weight_gradient_of_one_group_of_many_million_rows():
    """The bounds of a group's runs pass 32 bits on the way from 15.7 million rows on.  Small whole numbers: every partial
    sum is below 2^24, so the gradient is exact."""
    rows, m, k = (1 << 24) + 77, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda lo, hi: torch.randint(lo, hi, (rows, 64), generator=g, device="cuda", dtype=torch.int8).to(BF16)  # noqa: E731
    dy, x = draw(-1, 2), draw(-2, 3)
    codes = torch.empty(rows, k, dtype=U8, device="cuda")
    scales = torch.empty(k // 32, api.mx_scale_ld(rows), dtype=U8, device="cuda")
    api.moe_quantize_mxfp8(x, codes, scales)
    want = torch.zeros(m, k, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 20):
        want += dy[i:i + (1 << 20)].double().T @ x[i:i + (1 << 20)].double()
    ws = torch.empty(api.moe_grouped_wgrad_ckpt_workspace_size(1, rows, m, k), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dw = torch.full((1, m, k), 7.0, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, torch.tensor([0, rows], dtype=I32, device="cuda"), None, 1, dw, ws)
    assert api.moe_get_device_status(ws)[0] == 0
    assert torch.equal(dw[0].double(), want)


@pytest.mark.parametrize("n,d,e", [(8, 12544, 1001), (100, 65536, 17), (10000, 1024, 1024), (2000, 192, 1020),
                                   (45000, 128, 520), (1, 1152, 8), (600, 64, 1000)])
def test_router_backward_in_the_layers_own_scratch(n, d, e):
    """Workspaces without room for one partial product, or for those of all runs at a time.  Bounds: three bf16 terms hold
    the 24 bits of an entry, two lose 2^-17 of it; the tensor cores add 16 products at a time to an fp32 sum, each step
    off by less than 2^-23 of the magnitudes it has added, three chains; the terms', runs' and addend's sums 40 more."""
    g = torch.Generator().manual_seed(n + d + e)
    desc = api.make_desc(MoEConfig("case", n, d, 64, e, 1))
    size = api.moe_workspace_size(desc)[1]
    ws = torch.full((size + (1 << 20),), 0xab, dtype=U8, device="cuda")
    api.moe_workspace_init(ws[:size])
    dl = (torch.randn(n, e, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g)) * 1e-2).cuda()
    x, wg = torch.randn(n, d, generator=g).to(BF16).cuda(), (torch.randn(e, d, generator=g) * 0.1).to(BF16).cuda()
    dxi, dwi = torch.randn(n, d, generator=g).to(BF16).cuda(), torch.randn(e, d, generator=g).cuda()
    dx, dw = torch.full_like(dxi, 3.0), torch.full_like(dwi, 3.0)
    api.moe_router_backward(desc, dl, x, wg, dxi, dx, dwi, dw, ws[:size])
    dl64, x64, w64, dwi64 = dl.double(), x.double(), wg.double(), dwi.double()
    rx, mx = dxi.double() + dl64 @ w64, dl64.abs() @ w64.abs() + dxi.double().abs()
    assert ((dx.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + (2.0 ** -17 + (e / 8 + 8) * 2.0 ** -23) * mx
            * (1 + 2.0 ** -8)).all()
    rw, mw = dwi64 + dl64.T @ x64, dl64.abs().T @ x64.abs() + dwi64.abs()
    assert ((dw.double() - rw).abs() <= (3 * (n / 16 + 4) + 40) * 2.0 ** -23 * mw).all()
    dx2, dw2 = dxi.clone(), dwi.clone()
    api.moe_router_backward(desc, dl, x, wg, dx2, dx2, dw2, dw2, ws[:size])
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    api.moe_router_backward(desc, dl, x, wg, None, dx2, None, dw2, ws[:size])
    assert ((dw2.double() - (rw - dwi64)).abs() <= (3 * (n / 16 + 4) + 40) * 2.0 ** -23 * mw).all()
    assert api.moe_get_device_status(ws)[0] == 0 and (ws[size:] == 0xab).all()


def _rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def _quantised(v):
    codes = torch.empty(v.shape, dtype=U8, device="cuda")
    scales = torch.zeros(v.shape[1] // 32, api.mx_scale_ld(v.shape[0]), dtype=U8, device="cuda")
    api.moe_quantize_mxfp8(v, codes, scales)
    value = torch.empty_like(v)
    api.moe_dequantize_mxfp8(codes, scales, value)
    return codes, scales, value.double()


# What an addition to the tensor cores' fp32 accumulators does not hold is cut, about 1.5e-8 of the sum a step of 16
# elements: 3.7e-6 of the norm of a sum over 8192, in proportion to its length, 8e-6 where terms are few and alike.  Chains
# are kept short where an fp32 output hangs on them; these bounds lie between what the short chains leave (4.8e-7, 7e-7,
# 9e-7) and what one chain does.
@pytest.mark.parametrize("groups,off,m,k", [
    (1, [0, 8192], 192, 256), (1, [0, 8192], 1024, 2048), (2, [0, 8192, 16384], 1664, 1536),
    (16, [0, 100] + list(range(7200, 8192, 71)) + [8192], 1664, 1536)])
def test_weight_gradient_of_long_groups_is_summed_in_runs(groups, off, m, k):
    rows = off[-1]
    g = torch.Generator(device="cuda").manual_seed(rows + m)
    dy = torch.randn(rows, m, generator=g, device="cuda").to(BF16)
    codes, scales, x = _quantised(torch.randn(rows, k, generator=g, device="cuda").to(BF16))
    assert len(off) == groups + 1
    ws = torch.empty(api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, m, k), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dw = torch.full((groups, m, k), 7.0, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, torch.tensor(off, dtype=I32, device="cuda"), None, 1, dw, ws)
    for e in range(groups):
        r = slice(off[e], off[e + 1])
        assert _rel(dw[e], dy[r].double().T @ x[r]) <= 1e-6


@pytest.mark.parametrize("rows,d,f", [(200, 7168, 512), (1500, 7168, 1024), (4000, 7168, 2048)])
def test_gradient_of_row_weights_is_summed_in_chunks(rows, d, f):
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy = torch.randn(rows, d, generator=g, device="cuda").to(BF16)
    w2 = (torch.randn(1, d, f, generator=g, device="cuda") * 0.02).to(BF16)
    c1, s1, a1 = _quantised(torch.randn(rows, f, generator=g, device="cuda").to(BF16))
    c3, s3, a3 = _quantised(torch.randn(rows, f, generator=g, device="cuda").to(BF16))
    ws = torch.empty(api.moe_swiglu_backward_ckpt_workspace_size(1, rows, d, f), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    outs = [torch.empty(rows, f, dtype=BF16, device="cuda") for _ in range(3)]
    dg = torch.empty(rows, device="cuda")
    api.moe_swiglu_backward_ckpt(dy, torch.tensor([0, rows], dtype=I32, device="cuda"), w2, None, c1, s1, c3, s3, *outs,
                                 dg, ws)
    want = (dy.double() @ w2[0].double() * a1 * torch.sigmoid(a1) * a3).sum(1)
    assert _rel(dg, want) <= 1.5e-6


@pytest.mark.parametrize("n,d,e", [(4096, 1024, 256), (4096, 1088, 64), (4096, 704, 33), (4096, 1024, 8),
                                   (8000, 512, 16), (512, 1024, 64), (10000, 1024, 1024),
                                   (4096, 7168, 256), (16384, 7168, 8), (30000, 7168, 16)])
def test_router_weight_gradient_is_summed_in_runs(n, d, e):
    g = torch.Generator(device="cuda").manual_seed(n + e)
    desc = api.make_desc(MoEConfig("case", n, d, 64, e, 1))
    ws = torch.empty(api.moe_workspace_size(desc)[1], dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dl = torch.randn(n, e, generator=g, device="cuda") * 1e-3
    x = torch.randn(n, d, generator=g, device="cuda").to(BF16)
    wg = torch.randn(e, d, generator=g, device="cuda").to(BF16)
    dx, dw = torch.empty_like(x), torch.empty(e, d, device="cuda")
    api.moe_router_backward(desc, dl, x, wg, None, dx, None, dw, ws)
    assert _rel(dw, dl.double().T @ x.double()) <= 1.4e-6


@pytest.mark.parametrize("groups,long,rows,m,k", [(64, 8100, 8192, 1664, 1536), (40, 8192, 8192, 64, 64),
                                                  (100, 8000, 8192, 320, 128)])
def test_one_long_group_among_many_short_ones(groups, long, rows, m, k):
    """The same bound where the rows a group are few on average."""
    short = rows - long
    off = [short * e // (groups - 1) for e in range(groups)] + [rows]
    g = torch.Generator(device="cuda").manual_seed(rows + m)
    dy = torch.randn(rows, m, generator=g, device="cuda").to(BF16)
    codes, scales, x = _quantised(torch.randn(rows, k, generator=g, device="cuda").to(BF16))
    ws = torch.empty(api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, m, k), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dw = torch.full((groups, m, k), 7.0, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, torch.tensor(off, dtype=I32, device="cuda"), None, 1, dw, ws)
    for e in range(groups):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            assert not dw[e].any()
        else:
            assert _rel(dw[e], dy[r].double().T @ x[r]) <= 1e-6


def test_balance_of_a_checkpointing_layer_keeps_no_rows_of_its_own():
    """Beside what it writes (gradient of the logits, losses, counts) it holds nothing for the backward."""
    cfg = CONFIGS["small_softmax"]
    p = {key: None if v is None else v.cuda() for key, v in make_layer(cfg, "cpu").items()}
    layer = api.MoELayer(cfg, p, checkpoint=True)
    layer.forward(p["x"])
    off = torch.tensor([0, cfg.n_tok], dtype=I32, device="cuda")
    layer.balance_loss(off, 0.01)
    held = sum(v.numel() * v.element_size() for v in layer.balance.values() if isinstance(v, torch.Tensor))
    assert held <= 4 * (cfg.n_tok * cfg.n_exp + 2 + cfg.n_exp)
    got = layer.backward(make_dy(cfg, "cpu").cuda())
    x = torch.empty(cfg.n_tok, cfg.d_model, dtype=BF16, device="cuda")
    api.moe_dequantize_mxfp8(layer.ckpt["x"], layer.ckpt["x_scale"], x)
    with_loss = got["dw_gate"].clone()
    plain = layer.backward(make_dy(cfg, "cpu").cuda())["dw_gate"].double()      # the loss was taken back once
    want = plain + layer.balance["dlogits"].double().T @ x.double()
    assert _rel(with_loss, want) <= 1e-6
