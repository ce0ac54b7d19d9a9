"""The FP8 layer, the norm, the dropout and the quantisers at sizes where every
block of their grids takes several turns, against 64-bit formulas evaluated by
torch on the device.  The formulas are pinned to the CPU oracle first."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import BF16_TOL, np32
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig, make_dy, make_layer
from test_gpu_block import HALF, _check_norm, _desc, _norm
from test_gpu_fp8b import _check_layer

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------- 64-bit formulas
def _rows64(x):
    """The values that the 1 x 128 blocks of x (64 bits) stand for."""
    rows, cols = x.shape
    nb = -(-cols // 128)
    b = torch.nn.functional.pad(x, (0, nb * 128 - cols)).view(rows, nb, 128)
    s = b.abs().amax(2, keepdim=True).float() * torch.tensor(1.0 / 448.0, dtype=F32, device=x.device)
    s = torch.where(s > 0, s, torch.ones_like(s)).double()
    q = (b / s).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * s).view(rows, nb * 128)[:, :cols]


def _tile64(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return v * s


def _store(v):
    return v.float().to(BF16).double()


def _expert64(x, w1, w3, w2, dyw, xe):
    """One expert's y from the quantised rows x, and with the upstream dyw (as stored) its gradients."""
    a1, a3 = x @ w1.t(), x @ w3.t()
    h = a1 * torch.sigmoid(a1) * a3
    y = _rows64(h) @ w2.t()
    a1, a3, h = _store(a1), _store(a3), _store(h)
    dh = _rows64(dyw) @ w2
    sg = torch.sigmoid(a1)
    da1, da3 = _store(dh * a3 * sg * (1 + a1 * (1 - sg))), _store(dh * a1 * sg)
    dx = _rows64(da1) @ w1 + _rows64(da3) @ w3
    return y, dx, da1.t() @ xe, da3.t() @ xe, dyw.t() @ h


def _rel(a, b):
    d = float(b.norm())
    return float((a.double() - b).norm()) / d if d > 0 else float(a.double().norm())


def _check_rows(got, want, key):
    """Within the tolerance over all, and 99 rows in 100 within twice that of a typical row."""
    assert _rel(got, want) < BF16_TOL, (key, _rel(got, want))
    err = (got.double() - want).norm(dim=1) / want.norm(dim=1).square().mean().sqrt()
    assert float(torch.quantile(err, 0.99)) < 2 * BF16_TOL, key


def _check_layer64(cfg):
    p = make_layer(cfg, "cuda")
    dy = make_dy(cfg, "cuda")
    layer = api.MoELayer(cfg, p, train=True)
    out = layer.forward(p["x"]).clone()
    gr = layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status()[0] == 0
    wq, b = layer.w8q, layer.buf
    idx, w = b["topk_idx"].long(), b["topk_w"].double()
    x, d64 = p["x"].double(), dy.double()
    xq = _rows64(x)
    ref, dx, dg = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    for e in range(cfg.n_exp):
        tok, kk = torch.where(idx == e)
        if not tok.numel():
            assert not gr["dw1"][e].any() and not gr["dw3"][e].any() and not gr["dw2"][e].any()
            continue
        v = [_tile64(wq[k][e], wq[k + "_scale"][e]) for k in ("w1", "w3", "w2")]
        g = w[tok, kk][:, None]
        y, gx, dw1, dw3, dw2 = _expert64(xq[tok], *v, _store(d64[tok] * g), x[tok])
        ref.index_add_(0, tok, y * g)
        dx.index_add_(0, tok, _store(gx))
        dg[tok, kk] = (d64[tok] * _store(y)).sum(1)
        for key, want in (("dw1", dw1), ("dw3", dw3), ("dw2", dw2)):
            assert _rel(gr[key][e], want) < BF16_TOL, (key, e, tok.numel())
    if cfg.n_shared:
        v = [_tile64(wq[k], wq[k + "_scale"]) for k in ("ws1", "ws3", "ws2")]
        y, gx, dw1, dw3, dw2 = _expert64(xq, *v, d64, x)
        ref, dx = ref + y, dx + _store(gx)
        for key, want in (("dws1", dw1), ("dws3", dw3), ("dws2", dw2)):
            assert _rel(gr[key], want) < BF16_TOL, key
    dl = O.router_logit_grad(dg.cpu().numpy(), np32(b["topk_w"]), np32(b["logits"]), idx.cpu().numpy(), cfg.gate,
                             np.float64)
    dl = torch.from_numpy(dl).cuda()
    dx = dx + dl @ p["w_gate"].double()
    _check_rows(out, ref, "out")
    _check_rows(gr["dx"], dx, "dx")
    assert _rel(gr["dg"], dg) < BF16_TOL and _rel(gr["dw_gate"], dl.t() @ x) < BF16_TOL
    assert torch.equal(layer.forward(p["x"]).view(torch.int16), out.view(torch.int16))
    torch.cuda.empty_cache()


def test_formulas_are_the_oracles():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 272, generator=g) * torch.logspace(-3, 3, 272)[None]
    np.testing.assert_array_equal(_rows64(x.to(BF16).double().cuda()).cpu().numpy(),
                                  O.fp8_rows_value(x.to(BF16).float().numpy()))
    w = (torch.randn(1, 144, 272, generator=g) * 0.05).to(BF16)
    q = api.quantize_weights_fp8_tile({"w1": w.cuda()})
    np.testing.assert_array_equal(_tile64(q["w1"][0], q["w1_scale"][0]).cpu().numpy(),
                                  O.fp8_tile_value(q["w1"].cpu().numpy(), q["w1_scale"].cpu().numpy())[0])


@pytest.mark.parametrize("name", ["tiny", "small_sigmoid", "small_fine"])
def test_fp8b_layer_in_64_bits(name):
    _check_layer64(CONFIGS[name].replace(precision="fp8b"))


@pytest.mark.parametrize("tokens,d,f,shared", [(350, 256, 10304, 0), (350, 8256, 192, 0), (700, 1088, 4224, 4160)])
def test_fp8b_layer_several_tiles_a_block(tokens, d, f, shared):
    """Wide hidden layers and wide rows: above 152 tiles in the SwiGLU forward and backward products (8
    row tiles by 81 and by 41 column tiles), in the two-source product (8 by 33), and in the
    shared expert's (6 by 33 and by 17)."""
    cfg = MoEConfig("tiles", tokens, d, f, 4, 2, n_shared=1 if shared else 0, d_ff_shared=shared, precision="fp8b")
    _check_layer64(cfg)


def test_fp8b_layer_several_tiles_against_the_oracle():
    _check_layer(MoEConfig("tiles", 260, 320, 5184, 4, 2, n_shared=1, d_ff_shared=320, precision="fp8b"))


@pytest.mark.slow
@pytest.mark.parametrize("name", ["mixtral", "dsv3"])
def test_fp8b_layer_full_size(name):
    """Every token and every expert, forward and backward, in 64 bits."""
    torch.cuda.empty_cache()
    _check_layer64(CONFIGS[name].replace(precision="fp8b"))


# ------------------------------------------------------------------- quantisers
@pytest.mark.parametrize("rows,cols", [(40001, 144), (20003, 528)])
def test_quantise_rows_many(rows, cols):
    """More items than the grid has warps (152 x 32 blocks of 8)."""
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g) * torch.logspace(-3, 3, rows)[:, None]).to(BF16)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, api.fp8_scale_ld(cols), device="cuda")
    api.moe_quantize_fp8_rows(x.cuda(), codes, scales)
    rc, rs = O.fp8_rows_quantize(x.float().numpy())
    np.testing.assert_array_equal(scales[:, :rs.shape[1]].cpu().numpy().view(np.uint32), rs.view(np.uint32))
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)


def test_permute_fp8b_many_tokens():
    """Against the row quantiser, which the tests above hold to the oracle."""
    n, d, e, k = 20003, 576, 8, 2
    cfg = MoEConfig("many", n, d, 64, e, k, n_shared=1, d_ff_shared=64, precision="fp8b")
    desc = api.make_desc(cfg)
    ws = torch.empty(api.moe_workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(n, d, generator=g).to(BF16).cuda()
    idx = torch.stack([torch.randint(0, 4, (n,), generator=g), torch.randint(4, 8, (n,), generator=g)], 1).to(torch.int32)
    off = torch.zeros(e + 1, dtype=torch.int32)
    off[1:] = torch.bincount(idx.flatten(), minlength=e).cumsum(0)
    rows, copies = (torch.full((n * k,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    xp = torch.empty(n * k, d, dtype=BF16, device="cuda")
    xq, xqt = torch.empty(n * k, d, dtype=torch.uint8, device="cuda"), torch.empty(n, d, dtype=torch.uint8, device="cuda")
    ld = api.fp8_scale_ld(d)
    xs, xst = torch.full((n * k, ld), -1.0, device="cuda"), torch.full((n, ld), -1.0, device="cuda")
    api.moe_permute_fp8b(desc, x, idx.cuda(), off.cuda(), rows, copies, xp, xq, xs, xqt, xst, ws)
    assert api.moe_get_device_status(ws) == (0, 0)
    assert torch.equal(copies.long().sort().values, torch.arange(n * k, device="cuda"))
    tok = copies.long() // k
    assert torch.equal(xp, x[tok])
    codes, scales = torch.empty_like(xqt), torch.full_like(xst, -1.0)
    api.moe_quantize_fp8_rows(x, codes, scales)
    assert torch.equal(xqt, codes) and torch.equal(xst, scales)
    assert torch.equal(xq, codes[tok]) and torch.equal(xs, scales[tok])


# ------------------------------------------------------------------ norm, dropout
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("n,d", [(2433, 64), (5003, 320), (7001, 1024)])
def test_layernorm_backward_many_narrow_rows(n, d, kind):
    """More rows than 304 blocks of eight warps: every warp takes several."""
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(n, d, generator=g) * 2 + 0.5).to(kind).cuda()
    dres = torch.randn(n, d, generator=g).to(kind).cuda()
    dy = torch.randn(n, d, generator=g).to(BF16).cuda()
    gamma, beta = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    a = _norm(x, dy, gamma, beta, dres)
    _check_norm(x, dy, gamma, beta, dres, a)
    for u, v in zip(a, _norm(x, dy, gamma, beta, dres)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def _keep(seed, offset, n, p):
    """The oracle's keep mask for many elements: its steps on arrays of 64-bit integers."""
    m = np.uint64(0xFFFFFFFF)
    ctr = np.arange(-(-n // 4), dtype=np.uint64) + np.uint64(offset)
    c = [ctr & m, ctr >> np.uint64(32), np.zeros_like(ctr), np.zeros_like(ctr)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1)
    for i in (0, 1, len(words) - 1):
        assert words[i].tolist() == O.philox_words(seed, offset + i)
    return words.reshape(-1)[:n] >= np.uint64(int(p * 2.0 ** 32 + 0.5))


@pytest.mark.parametrize("kind", [BF16, F32])
def test_dropout_many_elements(kind):
    """Above 152 x 8 blocks of 256 threads' vectors, twice that for the backward's pairs."""
    n, d, k, p, rng = 1100, 4608, 3, 0.3, (987654321987, (1 << 32) - 1000)
    g = torch.Generator().manual_seed(4)
    rows = torch.randperm(n * k, generator=g).to(torch.int32)
    rows[5] = rows[n * k - 1] = -1
    y = torch.randn(n * k, d, generator=g).to(BF16).cuda()
    w = torch.softmax(torch.randn(n, k, generator=g), 1).cuda()
    ys = torch.randn(n, d, generator=g).to(BF16).cuda()
    res, dout = (torch.randn(n, d, generator=g).to(kind).cuda() for _ in range(2))
    desc, _ = _desc(n, d, k)
    r = torch.tensor(rng, dtype=torch.int64, device="cuda")
    out, dy = torch.empty_like(res), torch.empty(n, d, dtype=BF16, device="cuda")
    api.moe_combine_dropout(desc, y, rows.cuda(), w, ys, res, r, p, out)
    api.moe_dropout_backward(desc, dout, r, p, dy)
    keep = torch.from_numpy(_keep(*rng, n * d, p).reshape(n, d)).cuda()
    live = (rows >= 0).cuda().view(n, k, 1).double() * w.double()[:, :, None]
    yr = y.double()[rows.long().clamp_min(0).cuda()].view(n, k, d)
    total, mag = (yr * live).sum(1) + ys.double(), (yr.abs() * live).sum(1) + ys.double().abs()
    ref = res.double() + torch.where(keep, total / (1 - p), torch.zeros_like(total))
    tol = HALF[kind] * ref.abs() + (k + 5) * 2.0 ** -24 * (mag / (1 - p) + res.double().abs())
    assert ((out.double() - ref).abs() <= tol).all()
    assert torch.equal(out[~keep], res[~keep])
    rd = torch.where(keep, dout.double() / (1 - p), torch.zeros_like(ref))
    assert ((dy.double() - rd).abs() <= (2.0 ** -8 + 2.0 ** -22) * rd.abs()).all()
    assert not dy[~keep].any()
