"""GPU parity of the balance loss over sequences, the dense router gradient and the backward from activations kept in
8 bits, against 64-bit numpy, with bounds that count the roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import BF16_TOL, np32, rel, to_dev
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig, make_dy, make_layer

pytestmark = pytest.mark.gpu
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
U = 2.0 ** -24


def _ws(desc, which=1):
    ws = torch.empty(api.moe_workspace_size(desc)[which], dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    return ws


def _status(ws):
    return api.moe_get_device_status(ws)[0]


# ------------------------------------------------------------------ balance
def _balance(lg, idx, off, gate, coef=0.01, z=0.001, dloss=None, ws=None, stream=None, grad=True):
    n, e = lg.shape
    desc = api.make_desc(MoEConfig("case", n, 64, 64, e, idx.shape[1], gate=gate))
    ws = _ws(desc, 0) if ws is None else ws
    s = len(off) - 1
    counts = torch.full((s, e), -7, dtype=I32, device="cuda")
    loss = torch.full((2,), 9.0, device="cuda")
    dl = torch.full((n, e), 5.0, device="cuda") if grad else None
    api.moe_balance_loss(desc, lg, idx, torch.tensor(off, dtype=I32, device="cuda"), counts, loss, dl, ws, coef, z,
                         dloss, stream=stream)
    return counts, loss, dl, ws


def _check_balance(lg, idx, off, gate, got, coef=0.01, z=0.001, up=1.0):
    """An exponential of l - m carries the rounding of the difference (|l - m| U) and two ulps of its own, a
    sigmoid two such and its quotient, a sum over E / 32 terms a lane and five steps of a tree as many roundings: a
    probability is off by r = (E / 32 + 16 + 2 max|l|) U of itself, inner = sum f q by as much, and f - inner by r of
    (f + inner); the products add four roundings, lse is off by r + |lse| U."""
    counts, loss, dl, _ = got
    lg64, ih = lg.cpu().double().numpy(), idx.cpu().numpy()
    rc, rl, rg = O.balance_loss(lg64, ih, off, gate, coef, z)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    e = lg.shape[1]
    fin = np.where(np.isfinite(lg64), np.abs(lg64), 0.0).max()
    r = (e / 32 + 16 + 2 * fin) * U * 2
    assert abs(loss[0].item() - rl[0]) <= (r + U) * abs(rl[0])
    big = np.abs(lg64[np.isfinite(lg64)]).max() + np.log(e)
    assert abs(loss[1].item() - rl[1]) <= 2 * z * big * (r + big * U) + U * rl[1]
    if dl is None:
        return
    spans = np.diff(off)
    full, used = (spans > 0).sum(), spans[spans > 0].sum()
    tol = np.zeros_like(rg)
    for s, (a, b) in enumerate(zip(off, off[1:])):
        if b > a:
            f = rc[s] / (b - a)
            size = coef * e / full / (b - a) * (f + f.max()) + 2 * z / used * big   # the slopes are below 1
            tol[a:b] = size * (2 * r + 8 * U)
    assert (np.abs(np32(dl).astype(np.float64) - up * rg) <= abs(up) * tol + 1e-44).all()


def _routed(n, e, k, seed, scale=1.3):
    g = torch.Generator().manual_seed(seed)
    lg = (torch.randn(n, e, generator=g) * scale + 0.7 * torch.randn(e, generator=g)).cuda()
    return lg, lg.topk(k, dim=1).indices.to(I32)


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,e,k,off", [
    (1, 1, 1, [0, 1]), (1, 2, 2, [0, 1]), (5, 3, 1, [0, 0, 5, 5]), (33, 31, 4, [0, 7, 33]), (64, 32, 2, [0, 64]),
    (257, 33, 8, [4, 4, 5, 100, 100, 251]), (700, 60, 6, [0, 1, 2, 3, 699]), (2000, 64, 2, [0, 1000, 2000]),
    (1500, 129, 8, [0, 1500]), (3000, 256, 8, [10, 11, 2000, 2950]), (900, 300, 3, [0, 450, 900]),
    # one cluster, and the first sizes past it
    (256, 16, 2, [0, 256]), (64, 64, 8, [0, 10, 10, 40, 64]), (120, 33, 4, [3, 60, 60, 118]), (256, 8, 2, [0, 30, 31, 256]),
    (512, 8, 1, [0, 1, 2, 3, 4, 5, 6, 7, 512]), (512, 8, 1, [0, 1, 2, 3, 4, 5, 6, 7, 8, 512]), (257, 16, 2, [0, 257]),
    (63, 65, 8, [0, 63]), (400, 513, 32, [0, 399]), (350, 1024, 32, [0, 100, 350]), (20000, 8, 2, [0, 19999, 20000])])
def test_balance_loss(n, e, k, off, gate):
    lg, idx = _routed(n, e, k, n + e)
    got = _balance(lg, idx, off, gate)
    _check_balance(lg, idx, off, gate, got)
    assert _status(got[3]) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = _balance(lg, idx, off, gate, ws=got[3], stream=s)        # equal bits, the same workspace, another stream
    s.synchronize()
    for a, b in zip(got[:3], again[:3]):
        assert torch.equal(a.view(U8), b.view(U8))
    only = _balance(lg, idx, off, gate, ws=got[3], grad=False)       # without a gradient: the same losses
    assert torch.equal(only[1], got[1]) and torch.equal(only[0], got[0])


def test_balance_loss_many_sequences_and_scaled_gradient():
    n, e, k = 5000, 16, 2
    lg, idx = _routed(n, e, k, 1)
    cuts = np.sort(np.random.default_rng(2).integers(0, n, 4999))
    for off in ([0] + cuts.tolist() + [n], list(range(0, 5001))):
        up = torch.tensor([1024.0], device="cuda")
        got = _balance(lg, idx, off, "softmax", dloss=up)
        _check_balance(lg, idx, off, "softmax", got, up=1024.0)      # the losses themselves are not scaled


def test_balance_loss_is_the_auxiliary_loss_for_one_sequence():
    n, e, k = 600, 64, 4
    lg, idx = _routed(n, e, k, 3)
    desc = api.make_desc(MoEConfig("case", n, 64, 64, e, k))
    counts, loss, dl, ws = _balance(lg, idx, [0, n], "softmax", 0.01, 0.0)
    aux, da = torch.empty(1, device="cuda"), torch.empty(n, e, device="cuda")
    api.moe_aux_loss(desc, lg, counts[0].contiguous(), aux, da, ws, coef=0.01)
    assert loss[0].item() == pytest.approx(aux.item(), rel=2e-6) and loss[1].item() == 0
    assert (dl - da).abs().max() <= 1e-5 * da.abs().max()


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_balance_loss_masked_experts_and_extreme_logits(gate):
    n, e, k = 40, 48, 4
    lg, idx = _routed(n, e, k, 5)
    lg[3, 7], lg[4, :40], lg[5] = -float("inf"), -float("inf"), -float("inf")
    lg[6], lg[7, 2], lg[8] = torch.finfo(F32).min, 80.0, -80.0
    got = _balance(lg, idx, [0, n], gate, z=0.0)
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[1]).all()
    assert got[2][3, 7] == 0 and not got[2][4, :40].any() and not got[2][5].any()
    rc, rl, rg = O.balance_loss(np32(lg).astype(np.float64), idx.cpu().numpy(), [0, n], gate, 0.01, 0.0)
    keep = np.ones(n, bool)
    keep[6] = gate == "softmax"             # sigmoids of the lowest number are zero in 32 bits: no probability
    assert (np.abs(np32(got[2]) - rg)[keep] <= 200 * U * (np.abs(rg)[keep] + 0.01 * e / n)).all()
    np.testing.assert_array_equal(got[0].cpu().numpy(), rc)
    lg[9, 1], lg[10, 1] = float("nan"), float("inf")
    bad = _balance(lg, idx, [0, n], gate)
    assert torch.isnan(bad[2][9]).any() and torch.isnan(bad[1]).any()
    rest = [i for i in range(n) if i not in (9, 10, 6)]
    assert torch.isfinite(bad[2][rest]).all()                        # a row that is not finite keeps to itself


@pytest.mark.parametrize("n", [220, 300, 3000])      # one cluster for all, one block a sequence, a cluster of eight
def test_balance_loss_reports_offsets_and_indices(n):
    e, k = 16, 2
    lg, idx = _routed(n, e, k, 6)
    cut = _balance(lg, idx, [-5, 100, n + 9], "softmax")
    assert _status(cut[3]) == 4                                      # MOE_DEV_BAD_OFFSETS
    _check_balance(lg, idx, [0, 100, n], "softmax", cut)
    less = _balance(lg, idx, [0, 200, 100, n], "sigmoid")
    assert _status(less[3]) == 4
    assert not less[0].any() and not less[1].any() and not less[2].any()
    odd = idx.clone()
    odd[5, 0], odd[6, 1] = e, -1
    got = _balance(lg, odd, [0, n], "softmax")
    assert _status(got[3]) == 2                                      # MOE_DEV_BAD_INDEX
    good = torch.ones_like(odd, dtype=torch.bool)
    good[5, 0] = good[6, 1] = False
    assert torch.equal(got[0][0].cpu(), torch.bincount(odd[good].cpu(), minlength=e).to(I32))


def test_balance_loss_of_no_tokens():
    desc = api.make_desc(MoEConfig("case", 0, 64, 64, 8, 2))
    ws = _ws(desc, 0)
    counts, loss = torch.ones(3, 8, dtype=I32, device="cuda"), torch.ones(2, device="cuda")
    api.moe_balance_loss(desc, torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda"),
                         torch.zeros(4, dtype=I32, device="cuda"), counts, loss, None, ws)
    assert not counts.any() and not loss.any()
    lg, idx = _routed(20, 8, 2, 7)
    got = _balance(lg, idx, [20, 20, 20], "softmax")                 # tokens, but none in a sequence
    assert not got[0].any() and not got[1].any() and not got[2].any()


# ------------------------------------------------------------------- router
def _router(dl, x, wg, dxi, dwi, inplace=False, ws=None):
    n, e = dl.shape
    d = x.shape[1]
    desc = api.make_desc(MoEConfig("case", n, d, 64, e, 1))
    ws = _ws(desc) if ws is None else ws
    dx = dxi.clone() if inplace else torch.full((n, d), 3.0, dtype=BF16, device="cuda")
    dw = dwi.clone() if inplace else torch.full((e, d), 3.0, device="cuda")
    api.moe_router_backward(desc, dl, x, wg, dx if inplace else dxi, dx, dw if inplace else dwi, dw, ws)
    assert _status(ws) == 0
    return dx, dw


@pytest.mark.parametrize("n,d,e", [(1, 64, 1), (1, 128, 9), (7, 192, 8), (63, 64, 17), (130, 320, 60), (257, 512, 16),
                                   (129, 1088, 64), (256, 192, 33), (3, 128, 1024), (17, 448, 256), (40, 1024, 100), (70, 7168, 256), (512, 256, 65), (513, 256, 65), (1000, 448, 200), (2049, 576, 129), (300, 192, 1024),
                                   (3000, 704, 256), (4096, 2048, 8), (4096, 1088, 100)])
def test_router_backward(n, d, e):
    """Three bf16 terms hold the 24 bits of an entry, two lose 2^-17 of it.  The tensor cores add 16 products at a
    time to an fp32 sum, each step off by less than 2^-23 of the magnitudes it has added; the terms' sums, the runs'
    and dw_in a few more roundings; dx is rounded to bf16 once."""
    g = torch.Generator().manual_seed(n + d + e)
    dl = torch.randn(n, e, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g)) * 1e-2
    dl[n // 2] = 0.0
    dl = dl.cuda()
    x, wg = torch.randn(n, d, generator=g).to(BF16).cuda(), (torch.randn(e, d, generator=g) * 0.1).to(BF16).cuda()
    dxi, dwi = torch.randn(n, d, generator=g).to(BF16).cuda(), torch.randn(e, d, generator=g).cuda()
    dl64, x64, w64 = dl.cpu().double().numpy(), np32(x).astype(np.float64), np32(wg).astype(np.float64)
    mag_x, mag_w = np.abs(dl64) @ np.abs(w64), np.abs(dl64).T @ np.abs(x64)
    for a, b in ((dxi, dwi), (None, None)):
        dx, dw = _router(dl, x, wg, a, b)
        rx, rw = O.router_backward(dl64, x64, w64, 0.0 if a is None else np32(a).astype(np.float64),
                                   0.0 if b is None else np32(b).astype(np.float64))
        assert (np.abs(np32(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + (2.0 ** -17 + (e / 8 + 8) * 2.0 ** -23) * mag_x
                * (1 + 2.0 ** -8)).all()
        size = mag_w + (0 if b is None else np.abs(np32(b)))
        assert (np.abs(np32(dw).astype(np.float64) - rw) <= (3 * (n / 16 + 4) + 40) * 2.0 ** -23 * size).all()
    dx, dw = _router(dl, x, wg, dxi, dwi)
    ix, iw = _router(dl, x, wg, dxi, dwi, inplace=True)
    assert torch.equal(dx, ix) and torch.equal(dw, iw)


@pytest.mark.parametrize("n,d,e", [(1, 64, 2), (2, 4096, 3), (513, 64, 1), (514, 128, 9), (600, 192, 16), (5, 192, 5), (33, 1088, 1), (129, 64, 7), (500, 576, 2), (1001, 256, 4),
                                   (2600, 128, 16), (2047, 1984, 12), (3000, 1024, 8), (7000, 320, 3), (20000, 64, 9)])
def test_router_backward_of_few_experts(n, d, e):
    """Three bf16 terms of an entry are the entry but for 2^-24 of it, two (dx) but for 2^-17: a bf16 number is off by
    2^-9 of what it is made from at most, so what two leave is 2^-18 of it.  The tensor cores add 16 products at a time
    to an fp32 number, each step off by less than 2^-23 of the magnitudes it has added: two steps for dx, which is
    rounded to bf16 once; for a weight's gradient two for every 16 tokens, and 64 sums of warps, runs and the addend at most."""
    g = torch.Generator().manual_seed(n + d + e)
    dl = (torch.randn(n, e, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g)) * 1e-2).cuda()
    x, wg = torch.randn(n, d, generator=g).to(BF16).cuda(), (torch.randn(e, d, generator=g) * 0.1).to(BF16).cuda()
    dxi, dwi = torch.randn(n, d, generator=g).to(BF16).cuda(), torch.randn(e, d, generator=g).cuda()
    dl64, x64, w64 = dl.cpu().double().numpy(), np32(x).astype(np.float64), np32(wg).astype(np.float64)
    dx, dw = _router(dl, x, wg, dxi, dwi)
    rx, rw = O.router_backward(dl64, x64, w64, np32(dxi).astype(np.float64), np32(dwi).astype(np.float64))
    mag_x, mag_w = np.abs(dl64) @ np.abs(w64) + np.abs(np32(dxi)), np.abs(dl64).T @ np.abs(x64) + np.abs(np32(dwi))
    assert (np.abs(np32(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + (2.0 ** -17 + 2 * 2.0 ** -23) * mag_x * (1 + 2.0 ** -8)).all()
    assert (np.abs(np32(dw).astype(np.float64) - rw) <= (2 * (n / 16 + 1) + 64) * 2.0 ** -23 * mag_w).all()
    again = _router(dl, x, wg, dxi, dwi, inplace=True)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_router_backward_not_finite_and_no_tokens():
    n, d, e = 40, 128, 16
    g = torch.Generator().manual_seed(0)
    dl = torch.randn(n, e, generator=g).cuda()
    x, wg = torch.randn(n, d, generator=g).to(BF16).cuda(), torch.rand(e, d, generator=g).to(BF16).cuda() + 1
    clean, _ = _router(dl, x, wg, None, None)
    dl[3, 2], dl[4, 5] = float("inf"), float("nan")
    dx, dw = _router(dl, x, wg, None, None)
    assert torch.isinf(dx[3]).all() and torch.isnan(dx[4]).all()
    rest = [i for i in range(n) if i not in (3, 4)]
    assert torch.equal(dx[rest], clean[rest])
    assert torch.isnan(dw[5]).all() and torch.isfinite(dw[6]).all()
    empty = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    desc = api.make_desc(MoEConfig("case", 0, d, 64, e, 1))
    dwi, out = torch.randn(e, d, device="cuda"), torch.ones(e, d, device="cuda")
    for dw_in in (dwi, None):                    # no tokens: dw_in, or zero
        api.moe_router_backward(desc, empty(0, e), empty(0, d, dt=BF16), wg, None, empty(0, d, dt=BF16), dw_in, out,
                                _ws(desc))
        assert torch.equal(out, torch.zeros_like(out) if dw_in is None else dwi)


# -------------------------------------------------------------- kept rows
def _keep(v):
    """bf16 rows -> codes and scales of the library's quantiser."""
    rows, cols = v.shape
    codes = torch.empty(rows, cols, dtype=U8, device="cuda")
    scales = torch.full((cols // 32, api.mx_scale_ld(rows)), 255, dtype=U8, device="cuda")
    api.moe_quantize_mxfp8(v, codes, scales)
    return codes, scales


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 64), (100, 512), (33, 7168), (5000, 1024)])
def test_dequantize_is_exact(rows, cols):
    g = torch.Generator().manual_seed(rows)
    v = (torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))).to(BF16).cuda()
    v[0, :32] = 0.0
    codes, scales = _keep(v)
    out = torch.empty(rows, cols, dtype=BF16, device="cuda")
    api.moe_dequantize_mxfp8(codes, scales, out)
    np.testing.assert_array_equal(np32(out).astype(np.float64), O.kept_values(codes.cpu().numpy(), scales.cpu().numpy()))


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=U8).repeat(8).view(8, 256).cuda()
    scales = torch.randint(0, 255, (8, 16), generator=torch.Generator().manual_seed(1)).to(U8)
    scales[0, 0], scales[1, 1], scales[2, 2], scales[3, 3] = 0, 1, 246, 12
    out = torch.empty(8, 256, dtype=BF16, device="cuda")
    api.moe_dequantize_mxfp8(codes, scales.cuda(), out)
    want = O.kept_values(codes.cpu().numpy(), scales.numpy())
    with np.errstate(over="ignore"):
        want = torch.tensor(want).to(F32).to(BF16)          # rounds below bf16's range only, infinite above it
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


GROUPS = [  # groups, rows, offsets
    (1, 1, [0, 1]), (1, 200, [17, 150]), (3, 130, [0, 0, 129, 130]), (4, 300, [5, 5, 150, 151, 290]), (2, 257, [0, 128, 257]),
    (16, 777, None), (64, 500, None), (2, 1300, [0, 700, 1300])]


def _offsets(groups, rows, off, seed):
    if off is None:
        cut = np.sort(np.random.default_rng(seed).integers(0, rows + 1, groups - 1))
        off = [0] + cut.tolist() + [rows]
    return off


SWIGLU = [(g, r, o, d, f) for g, r, o in GROUPS for d, f in ((64, 64), (192, 320), (512, 256), (1088, 704))] + [
    # several chunks of the contraction; tiles of 64, 128 and 256 columns and pairs of 256
    (3, 300, [0, 10, 200, 300], 2624, 192), (2, 1900, None, 2688, 1024), (24, 4000, None, 1728, 1152),
    (2, 5000, [0, 2100, 4990], 2624, 1088), (1, 2600, [0, 2600], 7168, 2048)]


@pytest.mark.parametrize("groups,rows,off,d,f", SWIGLU)
def test_swiglu_backward(groups, rows, off, d, f):
    """dh is off by (D / 16 + 4) 2^-23 of its magnitudes sum |dy||w2|; the sigmoid's exponential (intrinsic: 2 + 1.2 |a1|
    ulps) and quotient give it 2^-18 for |a1| below 16, s + silu (1 - s) as much of 1 + |a1|; one rounding to
    bf16.  dg adds 128 terms a slice and the slices."""
    off = _offsets(groups, rows, off, rows)
    g = torch.Generator().manual_seed(rows + d + f)
    dy = torch.randn(rows, d, generator=g).to(BF16).cuda()
    w2 = (torch.randn(groups, d, f, generator=g) * 0.1).to(BF16).cuda()
    w = torch.rand(rows, generator=g).cuda()
    w[rows // 2] = 0.0                          # a weight of zero still has a gradient
    c1, s1 = _keep((torch.randn(rows, f, generator=g) * 1.5).to(BF16).cuda())
    c3, s3 = _keep(torch.randn(rows, f, generator=g).to(BF16).cuda())
    a1, a3 = (O.kept_values(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((c1, s1), (c3, s3)))
    assert np.abs(a1).max() < 16
    ws = torch.empty(api.moe_swiglu_backward_ckpt_workspace_size(groups, rows, d, f), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    outs = [torch.full((rows, f), 77.0, dtype=BF16, device="cuda") for _ in range(3)]
    dg = torch.full((rows,), 77.0, device="cuda")
    offs = torch.tensor(off, dtype=I32, device="cuda")
    api.moe_swiglu_backward_ckpt(dy, offs, w2, w, c1, s1, c3, s3, *outs, dg, ws)
    assert _status(ws) == 0
    dyh, w2h, wh = np32(dy).astype(np.float64), np32(w2).astype(np.float64), np32(w).astype(np.float64)
    want = O.swiglu_backward_kept(dyh, off, w2h, wh, a1, a3)
    lo, hi = off[0], off[-1]
    mag = np.zeros((rows, f))
    for e, (p, q) in enumerate(zip(off, off[1:])):
        mag[p:q] = np.abs(dyh[p:q]) @ np.abs(w2h[e])
    eh = (d / 16 + 4) * 2.0 ** -23 * mag
    s = O.train_step._sigmoid(a1)
    slope = np.abs(s * (1 + a1 * (1 - s)))
    size = [np.abs(a3) * slope, np.abs(a1 * s)]
    dh = want[1][lo:hi] / np.where(wh[lo:hi, None] * a1[lo:hi] * s[lo:hi] == 0, np.inf, wh[lo:hi, None] * a1[lo:hi]
                                   * s[lo:hi])
    for i, (o, r) in enumerate(zip(outs, want)):
        o = np32(o).astype(np.float64)
        assert (o[:lo] == 77).all() and (o[hi:] == 77).all()          # rows of no group are left alone
        o, r = o[lo:hi], r[lo:hi]
        tol = 2.0 ** -8 * np.abs(r) + 2.0 ** -17 * np.abs(r) + 1e-38
        if i == 0:
            tol += wh[lo:hi, None] * (size[0][lo:hi] * eh[lo:hi] + (mag * np.abs(a3) * s * (1 + 2 * np.abs(a1))
                                                                    * 2.0 ** -18)[lo:hi])
        elif i == 1:
            tol += wh[lo:hi, None] * size[1][lo:hi] * eh[lo:hi]
        assert (np.abs(o - r) <= tol).all(), i
    got = np32(dg).astype(np.float64)
    assert (got[:lo] == 77).all() and (got[hi:] == 77).all()
    act = np.abs(a1 * s * a3)
    tol = (eh * act).sum(1) + (2.0 ** -18 + (128 + 2 * np.ceil(f / 256)) * U) * (mag * act).sum(1)
    assert (np.abs(got - want[3]) <= tol)[lo:hi].all()
    # without weights (1) and without their gradient
    plain = [torch.full((rows, f), 77.0, dtype=BF16, device="cuda") for _ in range(3)]
    api.moe_swiglu_backward_ckpt(dy, offs, w2, torch.ones(rows, device="cuda"), c1, s1, c3, s3, *plain, None, ws)
    none = [torch.full((rows, f), 77.0, dtype=BF16, device="cuda") for _ in range(3)]
    api.moe_swiglu_backward_ckpt(dy, offs, w2, None, c1, s1, c3, s3, *none, None, ws)
    assert all(torch.equal(a, b) for a, b in zip(plain, none))


@pytest.mark.parametrize("groups,rows,off", GROUPS)
@pytest.mark.parametrize("m,k,top_k", [(64, 64, 1), (320, 192, 2), (256, 512, 4), (704, 1088, 3)])
def test_wgrad(groups, rows, off, m, k, top_k):
    """Kept values are bf16 numbers: only the sums round, 16 rows a step."""
    off = _offsets(groups, rows, off, rows)
    g = torch.Generator().manual_seed(rows + m + k)
    n = -(-rows // top_k)
    dy = torch.randn(rows, m, generator=g).to(BF16).cuda()
    codes, scales = _keep(torch.randn(n, k, generator=g).to(BF16).cuda())
    rmap = torch.randperm(n * top_k, generator=g)[:rows].to(I32).cuda()
    ws = torch.empty(api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, m, k), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dw = torch.full((groups, m, k), 7.0, device="cuda")
    offs = torch.tensor(off, dtype=I32, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, offs, rmap, top_k, dw, ws)
    assert _status(ws) == 0
    x = O.kept_values(codes.cpu().numpy(), scales.cpu().numpy())
    dyh = np32(dy).astype(np.float64)
    want = O.wgrad_kept(dyh, x, off, rmap.cpu().numpy(), top_k)
    mag = O.wgrad_kept(np.abs(dyh), np.abs(x), off, rmap.cpu().numpy(), top_k)
    steps = max(np.diff(off)) / 16 + 4
    assert (np.abs(np32(dw) - want) <= steps * 2.0 ** -23 * mag).all()
    for e in range(groups):
        if off[e] == off[e + 1]:
            assert not dw[e].any()
    if top_k == 1 and n == rows:                # no map: row r
        ident = torch.empty_like(dw)
        api.moe_grouped_wgrad_ckpt(dy, codes, scales, offs, None, 1, ident, ws)
        want = O.wgrad_kept(dyh, x, off, np.arange(rows), 1)
        mag = O.wgrad_kept(np.abs(dyh), np.abs(x), off, np.arange(rows), 1)
        assert (np.abs(np32(ident) - want) <= steps * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("groups,off", [(5, [0, 0, 9, 22, 23, 24]), (8, [0, 1, 1, 1, 7, 20, 20, 23, 24])])
@pytest.mark.parametrize("m,k", [(192, 12736), (12736, 192)])
def test_wgrad_of_few_rows_at_an_allocations_end(groups, off, m, k):
    """Rows of 128 KB or more in all, in groups of less that end with their allocations."""
    rows = off[-1]
    g = torch.Generator().manual_seed(groups + m)
    torch.cuda.empty_cache()
    need = api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, m, k)
    hold = [torch.empty(20 << 20, dtype=U8, device="cuda") for _ in range(2)]
    ws = hold[0][(20 << 20) - -(-need // 256) * 256:]
    api.moe_workspace_init(ws)
    dy = hold[1][(20 << 20) - 2 * rows * m:].view(BF16).view(rows, m)
    dy.copy_(torch.randn(rows, m, generator=g))
    codes, scales = _keep(torch.randn(rows, k, generator=g).to(BF16).cuda())
    dw = torch.full((groups, m, k), 7.0, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, torch.tensor(off, dtype=I32, device="cuda"), None, 1, dw, ws)
    assert _status(ws) == 0
    x, dyh = O.kept_values(codes.cpu().numpy(), scales.cpu().numpy()), np32(dy).astype(np.float64)
    want = O.wgrad_kept(dyh, x, off, np.arange(rows), 1)
    mag = O.wgrad_kept(np.abs(dyh), np.abs(x), off, np.arange(rows), 1)
    assert (np.abs(np32(dw) - want) <= (max(np.diff(off)) / 16 + 4) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("groups,rows,off,m,k", [
    (1, 5000, [0, 5000], 192, 256), (1, 4097, [0, 4097], 1024, 2048), (8, 4000, [0, 5, 5, 3000, 3100, 3500, 3500, 3990, 4000], 1664, 1536),
    (2, 6000, [3, 1795, 5990], 1664, 1536), (3, 8192, [0, 8192, 8192, 8192], 320, 704), (2, 1793, [0, 1793, 1793], 64, 64)])
def test_wgrad_of_long_groups(groups, rows, off, m, k):
    """Runs of 1792 rows at most: 112 steps of the tensor cores, each off by less than 2^-23 of the magnitudes it has
    added, and up to five sums of runs."""
    g = torch.Generator().manual_seed(rows + m)
    dy = torch.randn(rows, m, generator=g).to(BF16).cuda()
    codes, scales = _keep(torch.randn(rows, k, generator=g).to(BF16).cuda())
    ws = torch.empty(api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, m, k), dtype=U8, device="cuda")
    api.moe_workspace_init(ws)
    dw = torch.full((groups, m, k), 7.0, device="cuda")
    offs = torch.tensor(off, dtype=I32, device="cuda")
    api.moe_grouped_wgrad_ckpt(dy, codes, scales, offs, None, 1, dw, ws)
    assert _status(ws) == 0
    x, dyh = O.kept_values(codes.cpu().numpy(), scales.cpu().numpy()), np32(dy).astype(np.float64)
    want = O.wgrad_kept(dyh, x, off, np.arange(rows), 1)
    mag = O.wgrad_kept(np.abs(dyh), np.abs(x), off, np.arange(rows), 1)
    assert (np.abs(np32(dw) - want) <= (112 + 8) * 2.0 ** -23 * mag).all()
    again = torch.empty_like(dw)
    for _ in range(3):
        api.moe_grouped_wgrad_ckpt(dy, codes, scales, offs, None, 1, again, ws)
        assert torch.equal(again, dw)


def test_kept_products_report_offsets_and_indices():
    groups, rows, d, f = 3, 200, 64, 128
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(rows, d, generator=g).to(BF16).cuda()
    w2 = torch.randn(groups, d, f, generator=g).to(BF16).cuda()
    c, s = _keep(torch.randn(rows, f, generator=g).to(BF16).cuda())
    size = max(api.moe_swiglu_backward_ckpt_workspace_size(groups, rows, d, f),
               api.moe_grouped_wgrad_ckpt_workspace_size(groups, rows, d, f))

    def swiglu(off):
        ws = torch.zeros(size, dtype=U8, device="cuda")
        o = [torch.full((rows, f), 77.0, dtype=BF16, device="cuda") for _ in range(3)]
        dg = torch.full((rows,), 77.0, device="cuda")
        api.moe_swiglu_backward_ckpt(dy, torch.tensor(off, dtype=I32, device="cuda"), w2, None, c, s, c, s, *o, dg, ws)
        return o + [dg], _status(ws)

    def wgrad(off, rmap=None, div=1):
        ws = torch.zeros(size, dtype=U8, device="cuda")
        dw = torch.full((groups, d, f), 7.0, device="cuda")
        api.moe_grouped_wgrad_ckpt(dy, c, s, torch.tensor(off, dtype=I32, device="cuda"), rmap, div, dw, ws)
        return dw, _status(ws)
    good, bad = [0, 50, 120, rows], [-3, 50, 120, rows + 5]
    for a, b in zip(swiglu(good)[0], swiglu(bad)[0]):
        assert torch.equal(a, b)
    assert swiglu(bad)[1] == 4 and wgrad(bad)[1] == 4 and swiglu(good)[1] == 0
    assert torch.equal(wgrad(good)[0], wgrad(bad)[0])
    less = [0, 120, 50, rows]
    out, st = swiglu(less)
    assert st == 4 and all((o == 77).all() for o in out)
    dw, st = wgrad(less)
    assert st == 4 and not dw.any()
    ident = torch.arange(rows, dtype=I32, device="cuda")
    odd = ident.clone()
    odd[7], odd[60] = rows, -1
    dw, st = wgrad(good, odd)
    assert st == 2
    dz = dy.clone()
    dy[7] = dy[60] = 0.0                        # the rows that were not there
    assert torch.equal(dw, wgrad(good, ident)[0])
    dy.copy_(dz)


# ------------------------------------------------------------------ the layer
def _saved(layer, p, cfg):
    """The oracle's saved activations from what the layer kept."""
    k = {key: v.cpu().numpy() for key, v in layer.ckpt.items()}
    val = lambda key: O.kept_values(k[key], k[key + "_scale"])  # noqa: E731
    a1, a3 = val("a1"), val("a3")
    h = a1 * O.train_step._sigmoid(a1) * a3
    off, copy = layer.buf["offsets"].cpu().numpy(), layer.buf["copy_of_row"].cpu().numpy()
    experts = {}
    for e in range(cfg.n_exp):
        r = slice(off[e], off[e + 1])
        tok, kk = copy[r] // cfg.top_k, copy[r] % cfg.top_k
        experts[e] = (tok, kk, h[r] @ np32(p["w2"][e]).astype(np.float64).T, a1[r], a3[r], h[r])
    saved = {"experts": experts}
    if cfg.n_shared:
        b1, b3 = val("a1s"), val("a3s")
        hs = b1 * O.train_step._sigmoid(b1) * b3
        saved["shared"] = (None, b1, b3, hs)
    return saved, val("x")


@pytest.mark.parametrize("pair", ["0", "1", None])
@pytest.mark.parametrize("name", ["tiny", "small_softmax", "small_sigmoid", "small_fine"])
def test_layer_with_checkpoints_and_balance(name, pair, monkeypatch):
    """A training step of the two together: the forward's bits are the plain layer's, what is kept lies within half a
    code of the activations, and the gradients are those of the kept values."""
    if pair is not None:
        monkeypatch.setenv("MOE_GEMM_CTA_PAIR", pair)
    cfg = CONFIGS[name]
    p = to_dev(make_layer(cfg, "cpu"))
    dy = make_dy(cfg, "cpu").cuda()
    plain, layer = api.MoELayer(cfg, p), api.MoELayer(cfg, p, checkpoint=True)
    out = layer.forward(p["x"])
    assert torch.equal(out, plain.forward(p["x"]))
    for key in ("a1", "a3") + (("a1s", "a3s") if cfg.n_shared else ()):
        a = np32(plain.buf[key]).astype(np.float64)         # bf16 of the number that was encoded: 2^-8 off
        c, s = layer.ckpt[key].cpu().numpy(), layer.ckpt[key + "_scale"].cpu().numpy()
        scale = np.repeat(np.exp2(s[:, :len(a)].astype(np.float64) - 127).T, 32, axis=1)
        top = np.abs(a.reshape(len(a), -1, 32)).max(2) / scale[:, ::32]
        assert ((top > 255) & (top < 514)).all()            # 2^8 <= largest / scale < 2^9, off by 2^-8
        v = O.kept_values(c, s)
        tol = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * scale) * 1.01 + 2.0 ** -8 * np.abs(a)
        assert (np.abs(v - a) <= tol + np.maximum(np.abs(a) * 1.01 - 448 * scale, 0)).all()
    np.testing.assert_array_equal(layer.ckpt["x"].cpu().numpy(), O.mx_quantize(np32(p["x"]))[0])
    grads = {k: v.clone() for k, v in layer.backward(dy).items()}
    assert layer.device_status()[0] == 0
    saved, xk = _saved(layer, p, cfg)
    h = {k: (np32(v) if v is not None else None) for k, v in p.items()}
    idx, g = layer.buf["topk_idx"].cpu().numpy(), np32(layer.buf["topk_w"])
    lg = np32(layer.buf["logits"])
    shared = (h["ws1"], h["ws3"], h["ws2"]) if cfg.n_shared else None
    want = O.moe_backward(np32(dy), xk, lg, idx, g, h["w_gate"], h["w1"], h["w3"], h["w2"], saved, cfg.gate, shared,
                          dtype=np.float64)
    keys = ["dx", "dw_gate", "dw1", "dw3", "dw2", "dg"] + (["dws1", "dws3", "dws2"] if cfg.n_shared else [])
    for key in keys:
        assert rel(np32(grads[key]), want[key]) < BF16_TOL, key
    for e in range(cfg.n_exp):
        if layer.buf["offsets"][e] == layer.buf["offsets"][e + 1]:
            assert not grads["dw1"][e].any() and not grads["dw2"][e].any() and not grads["dw3"][e].any()

    # the balance loss of the same forward, in both layers: its gradient joins dx and dw_gate
    n = cfg.n_tok
    off = torch.tensor([0, n // 3, n // 3, n - 5], dtype=I32, device="cuda")
    for lay, x, base in ((layer, xk, grads), (plain, h["x"], None)):
        if base is None:
            base = {k: v.clone() for k, v in lay.backward(dy).items()}
        lay.forward(p["x"])
        loss = lay.balance_loss(off, 30.0, 10.0)
        full = lay.backward(dy)
        counts, rl, rg = O.balance_loss(lg, idx, off.tolist(), cfg.gate, 30.0, 10.0)
        np.testing.assert_array_equal(lay.balance["counts"].cpu().numpy(), counts)
        np.testing.assert_allclose(np32(loss), rl, rtol=1e-5)
        rx, rw = O.router_backward(rg, x, h["w_gate"], np32(base["dx"]), np32(base["dw_gate"]))
        assert rel(np32(full["dx"]), rx) < 2.0 ** -8 and rel(np32(full["dw_gate"]), rw) < 1e-5
        assert torch.equal(full["dw1"], base["dw1"])
        lay.forward(p["x"])                                 # a step without the loss: the plain gradients again
        again = lay.backward(dy)
        assert torch.equal(again["dx"], base["dx"]) and torch.equal(again["dw_gate"], base["dw_gate"])


def test_layer_of_no_tokens():
    cfg = CONFIGS["tiny"].replace(n_tok=0)
    p = to_dev(make_layer(cfg, "cpu"))
    layer = api.MoELayer(cfg, p, checkpoint=True, fused_dispatch=False)
    for v in layer.grads.values():
        v.fill_(3.0)
    state = {**{key: layer.buf[key] for key in ("logits", "topk_idx", "topk_w", "offsets", "row_of_copy", "copy_of_row")},
             **layer.ckpt}
    api.moe_grouped_ffn_ckpt(layer.desc, layer.buf["x_perm"], layer.buf["offsets"], p["x"], p, layer.ckpt,
                             layer.buf["y_perm"], None, layer.ws)
    api.moe_backward_ckpt(layer.desc, p["w_gate"], p, state, p["x"], layer.grads, layer.ws)
    assert not any(layer.grads[key].any() for key in ("dw1", "dw3", "dw2", "dw_gate"))


def test_layers_that_share_buffers():
    """A stack whose layers keep 8-bit rows of their own and share everything in passing."""
    cfg = CONFIGS["small_sigmoid"]
    ps = [to_dev(make_layer(cfg, "cpu")) for _ in range(3)]
    for i, p in enumerate(ps):
        p["w1"] = p["w1"].roll(i + 1, 1)
    dy = make_dy(cfg, "cpu").cuda()
    own = [api.MoELayer(cfg, p, checkpoint=True) for p in ps]
    first = api.MoELayer(cfg, ps[0], checkpoint=True)
    stack = [first] + [api.MoELayer(cfg, p, checkpoint=True, share=first) for p in ps[1:]]
    assert stack[2].ws is first.ws and stack[1].buf["x_perm"] is first.buf["x_perm"]
    x = {0: ps[0]["x"], 1: ps[0]["x"]}
    for i in range(3):
        for which, layers in enumerate((own, stack)):
            x[which] = layers[i].forward(x[which])
    assert torch.equal(x[0], x[1])
    g = {0: dy, 1: dy}
    for i in (2, 1, 0):
        for which, layers in enumerate((own, stack)):
            g[which] = layers[i].backward(g[which])["dx"]
    assert torch.equal(g[0], g[1])
    for a, b in zip(own, stack):
        for key in ("dw1", "dw3", "dw2", "dws1", "dw_gate", "dg"):
            assert torch.equal(a.grads[key], b.grads[key]), key
    with pytest.raises(ValueError, match="shares"):
        api.MoELayer(CONFIGS["tiny"], ps[0], checkpoint=True, share=first)
    with pytest.raises(ValueError, match="shares"):
        api.MoELayer(cfg, ps[0], share=first)


def test_captured_step_of_a_block_with_checkpoints_and_balance():
    cfg = CONFIGS["small_softmax"]
    p = to_dev(make_layer(cfg, "cpu"))
    n, d = cfg.n_tok, cfg.d_model
    gen = torch.Generator().manual_seed(5)
    gamma = torch.ones(d, device="cuda")
    x, dout = torch.randn(n, d, generator=gen).to(BF16).cuda(), torch.randn(n, d, generator=gen).to(BF16).cuda()
    off = torch.tensor([0, 300, n], dtype=I32, device="cuda")
    up = torch.tensor([8.0], device="cuda")
    block = api.MoEBlock(cfg, p, gamma, None, checkpoint=True)

    def step():
        block.forward(x)
        block.layer.balance_loss(off, 1.0, 0.1, dloss=up)
        return block.backward(dout)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(2):
        x.copy_(torch.randn(n, d, generator=gen).to(BF16))
        off[1] = 100 + i
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in block.layer.grads.items()}
        dx, loss = block.grads["dx"].clone(), block.layer.balance["loss"].clone()
        step()
        for key, v in block.layer.grads.items():
            assert torch.equal(v, got[key]), key
        assert torch.equal(dx, block.grads["dx"]) and torch.equal(loss, block.layer.balance["loss"])
    assert block.device_status()[0] == 0


def test_gradient_of_the_kept_backward_against_differences():
    """The loss sum(dy g y(a1, a3)) in 64 bits along a direction: a central difference of step 2^-10 is off by step^2
    times a third derivative of order one, each output by half a step of bf16 and dg by its sums."""
    rows, d, f, groups = 40, 64, 128, 2
    g = torch.Generator().manual_seed(9)
    off = [0, 25, 40]
    dy = torch.randn(rows, d, generator=g).to(BF16).cuda()
    w2 = (torch.randn(groups, d, f, generator=g) * 0.1).to(BF16).cuda()
    w = torch.rand(rows, generator=g).cuda()
    c1, s1 = _keep(torch.randn(rows, f, generator=g).to(BF16).cuda())
    c3, s3 = _keep(torch.randn(rows, f, generator=g).to(BF16).cuda())
    a1, a3 = (O.kept_values(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((c1, s1), (c3, s3)))
    ws = torch.zeros(api.moe_swiglu_backward_ckpt_workspace_size(groups, rows, d, f), dtype=U8, device="cuda")
    da1, da3, h = (torch.empty(rows, f, dtype=BF16, device="cuda") for _ in range(3))
    dg = torch.empty(rows, device="cuda")
    api.moe_swiglu_backward_ckpt(dy, torch.tensor(off, dtype=I32, device="cuda"), w2, w, c1, s1, c3, s3, da1, da3, h, dg,
                                 ws)
    dyh, w2h, wh = np32(dy).astype(np.float64), np32(w2).astype(np.float64), np32(w).astype(np.float64)

    def loss(u, v, ww):
        act = u * O.train_step._sigmoid(u) * v
        return sum((ww[a:b, None] * (act[a:b] @ w2h[e].T) * dyh[a:b]).sum() for e, (a, b) in enumerate(zip(off, off[1:])))
    r = np.random.default_rng(1)
    step = 2.0 ** -10
    for grad, vary in ((da1, 0), (da3, 1), (dg, 2)):
        args = [a1, a3, wh]
        v = r.standard_normal(args[vary].shape)
        at = lambda t: loss(*[q + t * v if i == vary else q for i, q in enumerate(args)])  # noqa: E731
        num = (at(step) - at(-step)) / (2 * step)
        got = np32(grad).astype(np.float64)
        assert abs(num - (got * v).sum()) <= (2.0 ** -8 * np.abs(got * v)).sum() + step ** 2 * np.abs(v ** 3).sum() * 10


class _User:
    """What one user of the entry points holds: inputs, a workspace for each call, outputs."""

    def __init__(self, seed, n=300, d=192, f=320, e=8, many=40, k=2):
        g = torch.Generator().manual_seed(seed)
        r = n * k
        self.lg, self.idx = _routed(n, e, k, seed)
        self.off = torch.tensor([0, 100 + seed, n], dtype=I32, device="cuda")
        self.desc = api.make_desc(MoEConfig("case", n, d, 64, e, k))
        self.wide = api.make_desc(MoEConfig("case", n, d, 64, many, k))
        rand = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
        self.x, self.wg, self.wgm, self.dx_in, self.dy = rand(n, d), rand(e, d), rand(many, d), rand(n, d), rand(r, d)
        self.w2, self.dlm = rand(e, d, f), torch.randn(n, many, generator=g).cuda()
        self.c, self.s = _keep(rand(r, f))
        self.cx, self.sx = _keep(self.x)
        self.rmap = torch.randint(0, r, (r,), generator=g).to(I32).cuda()   # rows more than once
        self.offs = torch.tensor(_offsets(e, r, None, seed), dtype=I32, device="cuda")
        size = [api.moe_workspace_size(self.desc)[1], api.moe_workspace_size(self.desc)[1], api.moe_workspace_size(self.wide)[1],
                api.moe_swiglu_backward_ckpt_workspace_size(e, r, d, f), api.moe_grouped_wgrad_ckpt_workspace_size(e, r, d, d)]
        self.ws = [torch.empty(b, dtype=U8, device="cuda") for b in size]
        for w in self.ws:
            api.moe_workspace_init(w)
        empty = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.out = dict(counts=empty(2, e, dt=I32), loss=empty(2, dt=F32), dl=empty(n, e, dt=F32), dx=empty(n, d),
                        dwg=empty(e, d, dt=F32), dxm=empty(n, d), dwm=empty(many, d, dt=F32), da1=empty(r, f), da3=empty(r, f),
                        h=empty(r, f), dg=empty(r, dt=F32), dw=empty(e, d, d, dt=F32), xd=empty(n, d))

    def run(self, stream=None):
        o = self.out
        api.moe_balance_loss(self.desc, self.lg, self.idx, self.off, o["counts"], o["loss"], o["dl"], self.ws[0], 0.01, 0.001,
                             None, stream=stream)
        api.moe_router_backward(self.desc, o["dl"], self.x, self.wg, self.dx_in, o["dx"], None, o["dwg"], self.ws[1],
                                stream=stream)
        api.moe_router_backward(self.wide, self.dlm, self.x, self.wgm, self.dx_in, o["dxm"], None, o["dwm"], self.ws[2],
                                stream=stream)
        api.moe_swiglu_backward_ckpt(self.dy, self.offs, self.w2, None, self.c, self.s, self.c, self.s, o["da1"], o["da3"],
                                     o["h"], o["dg"], self.ws[3], stream=stream)
        api.moe_grouped_wgrad_ckpt(self.dy, self.cx, self.sx, self.offs, self.rmap, 2, o["dw"], self.ws[4], stream=stream)
        api.moe_dequantize_mxfp8(self.cx, self.sx, o["xd"], stream=stream)

    def take(self):
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in self.out.items()}
        for v in self.out.values():
            v.zero_()
        torch.cuda.synchronize()
        return got


def test_entry_points_at_once_on_two_streams_and_captured():
    users = [_User(1), _User(2)]
    want = []
    for u in users:
        u.run()
        want.append(u.take())
        x = O.kept_values(u.cx.cpu().numpy(), u.sx.cpu().numpy())
        off, rmap, dy = u.offs.cpu().numpy(), u.rmap.cpu().numpy(), np32(u.dy).astype(np.float64)
        ref, mag = O.wgrad_kept(dy, x, off, rmap, 2), O.wgrad_kept(np.abs(dy), np.abs(x), off, rmap, 2)
        steps = np.diff(off).max() / 16 + 4
        assert (np.abs(np32(want[-1]["dw"]) - ref) <= steps * 2.0 ** -23 * mag).all()
    streams = [torch.cuda.Stream() for _ in users]
    for _ in range(5):
        for u, s in zip(users, streams):
            u.run(s)
    for u, w in zip(users, want):
        got = u.take()
        for key in w:
            assert torch.equal(got[key], w[key]), key
    graphs = []
    for u in users:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            u.run()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for u, w in zip(users, want):
        got = u.take()
        for key in w:
            assert torch.equal(got[key], w[key]), key
        assert all(_status(ws) == 0 for ws in u.ws)


def test_balance_loss_of_an_expert_chosen_twice():
    lg, _ = _routed(200, 12, 2, 3)
    idx = torch.full((200, 2), 5, dtype=I32, device="cuda")
    idx[::3] = 7
    _check_balance(lg, idx, [0, 90, 200], "softmax", _balance(lg, idx, [0, 90, 200], "softmax"))


@pytest.mark.parametrize("precision", ["mxfp8", "fp8w", "fp8b"])
def test_balance_loss_of_layers_on_other_operands(precision):
    """The loss's gradient joins dx and dw_gate of a step, and a step of other products follows with the same bits."""
    cfg = CONFIGS["small_softmax"].replace(precision=precision)
    p = to_dev(make_layer(cfg, "cpu"))
    dy = make_dy(cfg, "cpu").cuda()
    layer = api.MoELayer(cfg, p)
    layer.forward(p["x"])
    base = {k: v.clone() for k, v in layer.backward(dy).items()}
    off = torch.tensor([0, cfg.n_tok // 2, cfg.n_tok - 3], dtype=I32, device="cuda")
    layer.forward(p["x"])
    layer.balance_loss(off, 30.0, 10.0)
    full = layer.backward(dy)
    rg = O.balance_loss(np32(layer.buf["logits"]), layer.buf["topk_idx"].cpu().numpy(), off.tolist(), cfg.gate, 30.0, 10.0)[2]
    rx, rw = O.router_backward(rg, np32(p["x"]), np32(p["w_gate"]), np32(base["dx"]), np32(base["dw_gate"]))
    assert rel(np32(full["dx"]), rx) < 2.0 ** -8 and rel(np32(full["dw_gate"]), rw) < 1e-5
    layer.forward(p["x"])
    again = layer.backward(dy)
    assert all(torch.equal(again[k], v) for k, v in base.items())
    assert layer.device_status()[0] == 0


def test_captured_balance_loss_and_other_numbers_of_sequences():
    """A captured step goes on writing its own counts after calls with more sequences, and fewer."""
    cfg = CONFIGS["small_sigmoid"]
    p = to_dev(make_layer(cfg, "cpu"))
    n = cfg.n_tok
    layer = api.MoELayer(cfg, p)
    layer.forward(p["x"])
    two = torch.tensor([0, n // 2, n], dtype=I32, device="cuda")
    layer.balance_loss(two, 1.0, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(p["x"])
        layer.balance_loss(two, 1.0, 0.1)
    counts = layer.balance["counts"]
    graph.replay()
    torch.cuda.synchronize()
    want = counts.clone()
    many = torch.arange(0, n + 1, 3, dtype=I32, device="cuda")
    layer.balance_loss(many, 1.0, 0.1)
    other = layer.balance["counts"]
    kept = other.clone()
    assert other.shape[0] == len(many) - 1 and other.data_ptr() != counts.data_ptr()
    assert other.sum() == cfg.top_k * (many[-1] - many[0])
    counts.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(counts, want) and torch.equal(other, kept)
    loss = layer.balance_loss(two, 1.0, 0.1).clone()
    assert torch.equal(layer.balance["counts"], want) and torch.isfinite(loss).all()
