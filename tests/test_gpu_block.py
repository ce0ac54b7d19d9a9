"""GPU parity of the pre-norm block around the layer: layer norm and residual
dropout against 64-bit numpy, and the block that runs them with the layer."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import np32, rel, to_dev
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig, make_layer

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _desc(n, d, k=2):
    cfg = MoEConfig("block", n, d, 64, max(8, k), k)
    desc = api.make_desc(cfg)
    ws = torch.empty(api.moe_workspace_size(desc)[1], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    return desc, ws


def _norm(x, dy, gamma, beta, dres, eps=1e-5, stream=None):
    n, d = x.shape
    desc, ws = _desc(n, d)
    y = torch.empty(n, d, dtype=BF16, device="cuda")
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    dx, dgamma = torch.empty_like(x), torch.empty(d, device="cuda")
    dbeta = None if beta is None else torch.empty(d, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    api.moe_layernorm(desc, x, gamma, beta, y, mean, rstd, eps, stream=stream)
    api.moe_layernorm_backward(desc, dy, x, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream=stream)
    torch.cuda.synchronize()
    return y, mean, rstd, dx, dgamma, dbeta


def _check_norm(x, dy, gamma, beta, dres, got, eps=1e-5):
    """Sums of D terms: a thread adds 32 and a tree joins them, at most 32 + 32 roundings (2^-24
    each) of the terms' magnitude, so the mean is off by u max|x| with u = 64 * 2^-24, xhat by
    e = u (max|x| rstd + 4 max|xhat|) with the roundings of rstd and the products, and each later
    product by a few more; N rows add rows / 304 + 38 + 64 roundings."""
    y, mean, rstd, dx, dgamma, dbeta = got
    x64, dy64, g64 = np32(x).astype(np.float64), np32(dy).astype(np.float64), np32(gamma).astype(np.float64)
    b64 = None if beta is None else np32(beta).astype(np.float64)
    ry, rm, rr = O.layernorm(x64, g64, b64, eps)
    xhat = (x64 - rm[:, None]) * rr[:, None]
    u = 64 * 2.0 ** -24
    big = np.abs(x64).max(1)
    e = u * (big * rr + 4 * np.abs(xhat).max(1) + 1)[:, None]
    gm = np.abs(g64).max()
    assert (np.abs(np32(mean) - rm) <= u * big).all()
    # the variance feels the mean's error squared and 64 roundings of its own
    assert (np.abs(np32(rstd) - rr) <= rr * (u + (u * big * rr) ** 2)).all()
    assert (np.abs(np32(y) - ry) <= HALF[BF16] * np.abs(ry) + gm * e + 2.0 ** -22 * np.abs(ry)).all()
    rdx, rdg, rdb = O.layernorm_backward(dy64, x64, g64, eps, None if dres is None else np32(dres))
    gy = np.abs(dy64 * g64).max(1)[:, None]
    tol = HALF[x.dtype] * np.abs(rdx) + rr[:, None] * gy * (1 + np.abs(xhat)) * (e + u) * (2 + np.abs(xhat).max(1)[:, None])
    assert (np.abs(np32(dx) - rdx) <= tol + 2.0 ** -22 * np.abs(rdx)).all()
    adds = (x.shape[0] / 304 + 102) * 2.0 ** -24
    assert (np.abs(np32(dgamma) - rdg) <= adds * np.abs(dy64 * xhat).sum(0) + (np.abs(dy64) * e).sum(0)).all()
    if dbeta is not None:
        assert (np.abs(np32(dbeta) - rdb) <= adds * np.abs(dy64).sum(0)).all()


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d", [(1, 64), (3, 256), (9, 576), (310, 1024), (2, 1088), (5, 2560), (613, 4096), (7, 7168),
                                 (2, 8256), (3, 16384), (2, 32768)])
def test_layernorm(n, d, kind):
    g = torch.Generator().manual_seed(n + d)
    x = (torch.randn(n, d, generator=g) * 2 + 0.5).to(kind).cuda()
    dres = torch.randn(n, d, generator=g).to(kind).cuda()
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma, beta = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    a = _norm(x, dy, gamma, beta, dres)
    _check_norm(x, dy, gamma, beta, dres, a)
    s = torch.cuda.Stream()
    b = _norm(x, dy, gamma, beta, dres, stream=s)              # the same bits again, on another stream
    for u, v in zip(a, b):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    c = _norm(x, dy, gamma, None, None)                        # no bias, no residual
    _check_norm(x, dy, gamma, None, None, c)


def test_layernorm_large_mean_constant_rows_and_not_finite():
    g = torch.Generator().manual_seed(4)
    n, d = 6, 512
    x = torch.randn(n, d, generator=g) + 1000.0
    x[1] = 3.25                                                # no variance: rstd = 1 / sqrt(eps)
    x[2] = 0.0
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma = torch.ones(d, device="cuda")
    x = x.cuda()
    _check_norm(x, dy, gamma, None, None, _norm(x, dy, gamma, None, None))
    x[4, 7], x[5, 9] = float("inf"), float("nan")
    y, mean, rstd, dx, _, _ = _norm(x, dy, gamma, None, None)
    assert torch.isnan(y[4:]).all() and torch.isfinite(y[:4]).all() and torch.isfinite(dx[:4]).all()


@pytest.mark.parametrize("n,d", [(320, 2048), (330, 8192), (310, 8256), (160, 16448)])
def test_layernorm_large_mean_and_not_finite_beside_other_rows(n, d):
    """Rows that pass through a block together keep to themselves."""
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, d, generator=g) + 1000.0
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma = torch.ones(d, device="cuda")
    x = x.cuda()
    _check_norm(x, dy, gamma, None, None, _norm(x, dy, gamma, None, None))
    for kind in (F32, BF16):
        z = (x - 1000.0).to(kind)
        clean = _norm(z, dy, gamma, None, None)
        z[1, d - 1], z[n - 1, 0] = float("inf"), float("nan")
        y, mean, rstd, dx, _, _ = _norm(z, dy, gamma, None, None)
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[1] = bad[n - 1] = True
        assert torch.isnan(y[bad]).all()
        assert torch.equal(y[~bad], clean[0][~bad]) and torch.equal(dx[~bad], clean[3][~bad])


def test_layernorm_without_tokens_clears_the_weight_gradients():
    desc, ws = _desc(1, 128)
    desc.n_tok = 0
    dg, db = torch.ones(128, device="cuda"), torch.ones(128, device="cuda")
    e = torch.empty(0, 128, dtype=BF16, device="cuda")
    m = torch.empty(0, device="cuda")
    api.moe_layernorm_backward(desc, e, e, dg, m, m, None, e, dg, db, ws)
    assert not dg.any() and not db.any()


def _combine(n, d, k, kind, shared, p, seed, resid=True, drop=(), rng=(3, 11)):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randperm(n * k, generator=g).to(torch.int32)
    for c in drop:
        rows[c] = -1                                           # a copy dropped by a capacity
    y = torch.randn(n * k, d, generator=g).to(BF16)
    w = torch.softmax(torch.randn(n, k, generator=g), 1)
    ys = torch.randn(n, d, generator=g).to(BF16) if shared else None
    res = torch.randn(n, d, generator=g).to(kind) if resid else None
    desc, _ = _desc(n, d, k)
    out = torch.empty(n, d, dtype=kind, device="cuda")
    r = torch.tensor(rng, dtype=torch.int64, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    api.moe_combine_dropout(desc, dev(y), dev(rows), dev(w), dev(ys), dev(res), r, p, out)
    torch.cuda.synchronize()
    w64 = w.double().numpy().copy().reshape(-1)
    w64[rows.numpy() < 0] = 0.0
    yr = y.double().numpy()[rows.long().clamp_min(0).numpy()].reshape(n, k, d)
    w64 = w64.reshape(n, k, 1)
    total, mag = (yr * w64).sum(1), (np.abs(yr) * w64).sum(1)
    if shared:
        total, mag = total + ys.double().numpy(), mag + np.abs(ys.double().numpy())
    keep = O.dropout_keep(rng[0], rng[1], n * d, p).reshape(n, d)
    base = res.double().numpy() if resid else np.zeros((n, d))
    ref = base + np.where(keep, total / (1 - p), 0.0)
    # K + 1 additions, the factor and its product, the residual sum: 2^-24 of the magnitudes each
    tol = HALF[kind] * np.abs(ref) + (k + 5) * 2.0 ** -24 * (mag / (1 - p) + np.abs(base))
    got = np32(out)
    assert (np.abs(got - ref) <= tol).all()
    # where nothing is kept the residual passes untouched
    np.testing.assert_array_equal(got[~keep], np.float32(base)[~keep])
    return desc, r, keep


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d,k,shared,p", [(1, 64, 1, False, 0.1), (3, 64, 2, True, 0.5), (37, 128, 3, True, 0.0),
                                            (5, 704, 8, False, 0.3), (13, 192, 6, True, 0.999999)])
def test_combine_dropout(n, d, k, shared, p, kind):
    desc, r, keep = _combine(n, d, k, kind, shared, p, n + d)
    dout = torch.randn(n, d).to(kind).cuda()
    dy = torch.empty(n, d, dtype=BF16, device="cuda")
    api.moe_dropout_backward(desc, dout, r, p, dy)
    ref = np.where(keep, np32(dout).astype(np.float64) / (1 - p), 0.0)
    assert (np.abs(np32(dy) - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref)).all()
    assert not np32(dy)[~keep].any()


def test_combine_dropout_without_residual_dropped_copies_and_wide_counters():
    _combine(4, 128, 2, BF16, False, 0.25, 5, resid=False)
    _combine(4, 128, 2, F32, True, 0.25, 6, drop=(0, 1, 5))    # token 0 has no copy left
    # seed and counter past 32 bits, and a counter that wraps
    _combine(3, 64, 2, F32, False, 0.5, 7, rng=((1 << 62) + 12345, (1 << 32) - 3))
    _combine(3, 64, 2, F32, False, 0.5, 8, rng=(-2, -5))


def test_combine_dropout_passes_nothing_of_a_dropped_nan():
    n, d = 2, 64
    desc, _ = _desc(n, d, 1)
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    y = torch.full((n, d), float("nan"), dtype=BF16, device="cuda")
    out = torch.empty(n, d, device="cuda")
    res = torch.ones(n, d, device="cuda")
    api.moe_combine_dropout(desc, y, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.ones(n, 1).cuda(),
                            None, res, rng, 0.5, out)
    keep = torch.from_numpy(O.dropout_keep(1, 2, n * d, 0.5).reshape(n, d)).cuda()
    assert torch.isnan(out[keep]).all() and (out[~keep] == 1).all()


@pytest.mark.parametrize("precision", ["bf16", "fp8b", "mxfp8"])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_block_is_its_parts(precision, kind):
    cfg = CONFIGS["small_sigmoid"].replace(precision=precision)
    p = to_dev(make_layer(cfg, "cpu"))
    g = torch.Generator().manual_seed(8)
    n, d = cfg.n_tok, cfg.d_model
    gamma, beta = (1 + 0.1 * torch.randn(d, generator=g)).cuda(), torch.randn(d, generator=g).cuda()
    x, dout = (torch.randn(n, d, generator=g).to(kind).cuda() for _ in range(2))
    block = api.MoEBlock(cfg, p, gamma, beta, p=0.2, seed=99, stream_dtype=kind)
    first = block.forward(x).clone()
    out = block.forward(x).clone()                             # the second draw
    grads = block.backward(dout)
    torch.cuda.synchronize()
    assert block.device_status()[0] == 0
    assert not torch.equal(first, out)
    # by its parts: the layer of the normed input, the mask of the second call
    ry, _, _ = O.layernorm(np32(x), np32(gamma).astype(np.float64), np32(beta), 1e-5)
    assert rel(np32(block.normed), ry) < 2.0 ** -8
    layer = api.MoELayer(cfg, p, train=True)
    moe = np32(layer.forward(block.normed)).astype(np.float64)
    keep = O.dropout_keep(99, (n * d + 3) // 4, n * d, 0.2).reshape(n, d)
    ref = np32(x) + np.where(keep, moe / 0.8, 0.0)
    # the layer's own output is rounded to bf16 (2^-8 of it) where the block's is not
    assert (np.abs(np32(out) - ref) <= HALF[kind] * np.abs(ref) + (2.0 ** -8 + 2.0 ** -20) * np.abs(moe) / 0.8 + 1e-6).all()
    dmoe = np.where(keep, np32(dout).astype(np.float64) / 0.8, 0.0)
    assert rel(np32(block.dmoe), dmoe) < 2.0 ** -8
    inner = layer.backward(block.dmoe)
    for key in ("dw1", "dw2", "dw_gate", "dx"):
        assert torch.equal(grads["layer"][key], inner[key])
    dx, dg, db = O.layernorm_backward(np32(inner["dx"]), np32(x), np32(gamma).astype(np.float64), 1e-5, np32(dout))
    assert rel(np32(grads["dx"]), dx) < 2.0 ** -8
    assert rel(np32(grads["dgamma"]), dg) < 1e-5 and rel(np32(grads["dbeta"]), db) < 1e-5
    # inference drops nothing and moves no counter
    quiet = api.MoEBlock(cfg, p, gamma, beta, p=0.2, train=False, stream_dtype=kind)
    q = np32(quiet.forward(x))
    assert (np.abs(q - (np32(x) + moe)) <= HALF[kind] * np.abs(q) + (2.0 ** -8 + 2.0 ** -20) * np.abs(moe) + 1e-6).all()
    assert quiet.rng.tolist() == [0, 0]


def test_block_captured_step_draws_anew_at_each_replay():
    cfg = CONFIGS["tiny"].replace(precision="fp8b", d_model=128)
    p = to_dev(make_layer(cfg, "cpu"))
    n, d = cfg.n_tok, cfg.d_model
    gamma = torch.ones(d, device="cuda")
    x, dout = torch.randn(n, d).to(BF16).cuda(), torch.randn(n, d).to(BF16).cuda()
    block = api.MoEBlock(cfg, p, gamma, None, p=0.5, seed=7)

    def step():
        block.forward(x)
        block.backward(dout)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    per = (n * d + 3) // 4
    for i in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        keep = O.dropout_keep(7, i * per, n * d, 0.5).reshape(n, d)
        assert not np32(block.dmoe)[~keep].any()
        np.testing.assert_array_equal(np32(block.out)[~keep], np32(x)[~keep])
        assert (np32(block.dmoe)[keep] == 2 * np32(dout)[keep]).all()
    assert block.device_status()[0] == 0


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d", [(305, 1088), (611, 2048), (400, 2560), (1000, 4096), (307, 7168), (330, 8192)])
def test_layernorm_many_rows(n, d, kind):
    """More rows than blocks: every block takes several, through all its row buffers."""
    g = torch.Generator().manual_seed(n + d + 1)
    x = (torch.randn(n, d, generator=g) * 2 - 0.5).to(kind).cuda()
    dres = torch.randn(n, d, generator=g).to(kind).cuda()
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma, beta = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    a = _norm(x, dy, gamma, beta, dres)
    _check_norm(x, dy, gamma, beta, dres, a)
    for u, v in zip(a, _norm(x, dy, gamma, beta, dres)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    _check_norm(x, dy, gamma, None, None, _norm(x, dy, gamma, None, None))


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d", [(153, 8256), (400, 9024), (311, 12288), (160, 16384), (77, 16448), (154, 24576),
                                 (80, 32768)])
def test_layernorm_wide_rows(n, d, kind):
    """Rows that two or four blocks share, several a cluster; the last block's share may be smaller."""
    g = torch.Generator().manual_seed(n + d + 2)
    x = (torch.randn(n, d, generator=g) * 2 - 0.5).to(kind).cuda()
    dres = torch.randn(n, d, generator=g).to(kind).cuda()
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma, beta = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    a = _norm(x, dy, gamma, beta, dres)
    _check_norm(x, dy, gamma, beta, dres, a)
    for u, v in zip(a, _norm(x, dy, gamma, beta, dres)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    _check_norm(x, dy, gamma, None, None, _norm(x, dy, gamma, None, None))


def test_layernorm_gradient_against_differences():
    """The loss sum(y t) in 64 bits along a direction against the kernel's gradients: a central
    difference of step 2^-10 is off by step^2 times the third derivative (order one), and
    the gradients by the roundings of the checks above."""
    g = torch.Generator().manual_seed(11)
    n, d = 4, 1536
    x, v = torch.randn(n, d, generator=g), torch.randn(n, d, generator=g)
    t = torch.randn(n, d, generator=g).to(BF16)
    gamma, beta, vg = (torch.randn(d, generator=g) for _ in range(3))
    _, _, _, dx, dgamma, dbeta = _norm(x.cuda(), t.cuda(), gamma.cuda(), beta.cuda(), None)
    x64, g64, b64, t64 = (np32(w).astype(np.float64) for w in (x, gamma, beta, t))
    loss = lambda xx, gg: (O.layernorm(xx, gg, b64, 1e-5)[0] * t64).sum()  # noqa: E731
    h = 2.0 ** -10
    vx, vgn = np32(v).astype(np.float64), np32(vg).astype(np.float64)
    num_x = (loss(x64 + h * vx, g64) - loss(x64 - h * vx, g64)) / (2 * h)
    num_g = (loss(x64, g64 + h * vgn) - loss(x64, g64 - h * vgn)) / (2 * h)
    scale = np.sqrt(n * d)
    assert abs(num_x - (np32(dx).astype(np.float64) * vx).sum()) <= 1e-4 * scale
    assert abs(num_g - (np32(dgamma).astype(np.float64) * vgn).sum()) <= 1e-4 * scale
    assert abs(np32(dbeta).astype(np.float64) - t64.sum(0)).max() <= 4 * 2.0 ** -24 * np.abs(t64).sum(0).max()
