"""GPU parity of the FP8 products with one fp32 scale per block of 128: the row
quantiser bit for bit, the grouped product and the layer against 64-bit
numpy on the same codes."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import BF16_TOL, host_params, np32, rel, routing_agreement, to_dev
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig, make_dy, make_layer

pytestmark = pytest.mark.gpu
BAD_OFFSETS = 4


def _quantise(x):
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.full((x.shape[0], api.fp8_scale_ld(x.shape[1])), -1.0, device="cuda")
    api.moe_quantize_fp8_rows(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (7, 144), (33, 1040), (5, 2560)])
def test_quantise_rows_bitexact(rows, cols):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=g) * torch.logspace(-8, 8, cols)[None]).to(torch.bfloat16)
    x[0, : cols // 2] = 0.0
    codes, scales = _quantise(x)
    rc, rs = O.fp8_rows_quantize(x.float().numpy())
    nb = rs.shape[1]
    np.testing.assert_array_equal(scales[:, :nb].cpu().numpy().view(np.uint32), rs.view(np.uint32))
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    assert (scales[:, nb:] == -1.0).all()                  # nothing past the blocks is written


def test_quantise_rows_every_bf16_value_on_every_border():
    # one block per amax, holding 127 of all finite bf16 magnitudes: borders between two codes included
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    vals = (bits << 16).view(torch.float32)
    vals = torch.cat([vals, -vals])
    for amax in (448.0, 1.0, 3.0, 0.0107421875, 2.0 ** -120, 3.0e38, 1e-38, 1e-40):
        v = vals[vals.abs() <= amax]
        if not v.numel():
            continue
        v = torch.nn.functional.pad(v, (0, -v.numel() % 127)).view(-1, 127)
        x = torch.cat([torch.full((v.shape[0], 1), amax), v], 1).to(torch.bfloat16)
        codes, scales = _quantise(x)
        rc, rs = O.fp8_rows_quantize(x.float().numpy())
        np.testing.assert_array_equal(scales[:, :1].cpu().numpy().view(np.uint32), rs.view(np.uint32), str(amax))
        np.testing.assert_array_equal(codes.cpu().numpy(), rc, str(amax))


def test_quantise_rows_not_finite():
    x = torch.randn(3, 256).to(torch.bfloat16)
    x[0, 5], x[1, 130] = float("nan"), float("inf")
    codes, scales = _quantise(x)
    assert codes[0, 5] & 0x7F == 0x7F and (codes[0, 128:] & 0x7F != 0x7F).all()
    assert torch.isinf(scales[1, 1]) and codes[1, 130] & 0x7F == 0x7F
    rc, _ = O.fp8_rows_quantize(x[2:].float().numpy())
    np.testing.assert_array_equal(codes[2:].cpu().numpy(), rc)


def _weights(g, e, r, c):
    w = (torch.randn(e, r, c, generator=g) * 0.05).to(torch.bfloat16).cuda()
    q = api.quantize_weights_fp8_tile({"w1": w})
    return q["w1"], q["w1_scale"]


def _product_ref(codes, scales, off, w, ws, mn):
    a = O.fp8_rows_dequantize(codes.cpu().numpy(), scales[:, : -(-codes.shape[1] // 128)].cpu().numpy())
    b = O.fp8_tile_value(w.cpu().numpy(), ws.cpu().numpy())
    if not mn:
        b = b.transpose(0, 2, 1)
    out, mag = np.zeros((a.shape[0], b.shape[2])), np.zeros((a.shape[0], b.shape[2]))
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        out[lo:hi] = a[lo:hi] @ b[e]
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(b[e])
    return out, mag


def _product_tol(ref, mag, k):
    """bf16 store: half a step; the sum: within a block up to 128 additions that may truncate
    (2^-23 of the magnitude each), across blocks one rounding (2^-24) for each of the nb
    additions and three for the scales."""
    return 2.0 ** -8 * np.abs(ref) + (128 * 2.0 ** -23 + (k // 128 + 4) * 2.0 ** -24) * mag


GROUPS = [[1], [0], [5, 0, 130], [128, 128], [127, 129, 1, 0, 300, 0], [0, 0, 0, 257]]


@pytest.mark.parametrize("mn", [False, True])
@pytest.mark.parametrize("n,k", [(16, 16), (64, 128), (144, 272), (256, 384), (400, 1168), (528, 128)])
def test_grouped_product(n, k, mn):
    for i, sizes in enumerate(GROUPS):
        g = torch.Generator().manual_seed(i + n + k)
        rows = sum(sizes)
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        x = torch.randn(max(rows, 1), k, generator=g).to(torch.bfloat16)[:rows]
        w, ws = _weights(g, len(sizes), *((k, n) if mn else (n, k)))
        if rows == 0:
            continue
        codes, scales = _quantise(x)
        out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
        work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(len(sizes), rows, n, k), dtype=torch.uint8,
                           device="cuda")
        api.moe_workspace_init(work)
        for _ in range(2):                                 # a workspace is ready for the next call
            api.moe_grouped_gemm_fp8(codes, scales, torch.from_numpy(off).cuda(), w, ws, out, work, b_mn=mn)
        assert api.moe_get_device_status(work) == (0, 0)
        ref, mag = _product_ref(codes, scales, off, w, ws, mn)
        err = np.abs(np32(out) - ref)
        assert (err <= _product_tol(ref, mag, k)).all(), (sizes, float((err - _product_tol(ref, mag, k)).max()))


@pytest.mark.parametrize("mn", [False, True])
@pytest.mark.parametrize("sizes,n,k", [([8], 144, 2048), ([1, 0, 130], 512, 2064), ([3, 40], 1040, 4112),
                                       ([300], 272, 8208), ([1], 4112, 1168), ([0, 129, 0], 16, 16400)])
def test_grouped_product_split_along_the_contraction(sizes, n, k, mn):
    """Few tiles: clusters of CTAs share each.  At most nb / ranks + ranks <= nb additions a sum."""
    g = torch.Generator().manual_seed(n + k)
    rows = sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    x = torch.randn(rows, k, generator=g).to(torch.bfloat16)
    w, ws = _weights(g, len(sizes), *((k, n) if mn else (n, k)))
    codes, scales = _quantise(x)
    work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(len(sizes), rows, n, k), dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(work)
    outs = []
    for _ in range(3):
        out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
        api.moe_grouped_gemm_fp8(codes, scales, torch.from_numpy(off).cuda(), w, ws, out, work, b_mn=mn)
        outs.append(out)
    assert api.moe_get_device_status(work) == (0, 0)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])   # the same order every time
    ref, mag = _product_ref(codes, scales, off, w, ws, mn)
    assert (np.abs(np32(outs[0]) - ref) <= _product_tol(ref, mag, k)).all()


def test_grouped_product_rows_of_no_group_and_offsets_past_the_rows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 128, generator=g).to(torch.bfloat16)
    codes, scales = _quantise(x)
    w, ws = _weights(g, 2, 64, 128)
    for off, status in (([3, 10, 30], 0), ([0, 20, 4000], BAD_OFFSETS), ([-5, 20, 40], BAD_OFFSETS)):
        out = torch.full((40, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(2, 40, 64, 128), dtype=torch.uint8, device="cuda")
        api.moe_workspace_init(work)
        api.moe_grouped_gemm_fp8(codes, scales, torch.tensor(off, dtype=torch.int32, device="cuda"), w, ws, out, work)
        assert api.moe_get_device_status(work)[0] == status
        cut = np.clip(off, 0, 40)
        ref, mag = _product_ref(codes, scales, cut, w, ws, False)
        inside = np.zeros(40, bool)
        inside[cut[0]:cut[2]] = True
        assert (np32(out)[~inside] == 7.0).all()
        assert (np.abs(np32(out) - ref) <= _product_tol(ref, mag, 128))[inside].all()


def test_split_product_descending_offsets_are_flagged():
    """More tiles than ascending offsets over these rows could have: those past the launch's clusters are left out."""
    g = torch.Generator().manual_seed(5)
    n, k = 144, 2048
    codes, scales = _quantise(torch.randn(300, k, generator=g).to(torch.bfloat16))
    w, ws = _weights(g, 5, n, k)
    out = torch.empty(300, n, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(5, 300, n, k), dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(work)
    off = torch.tensor([0, 300, 0, 300, 0, 300], dtype=torch.int32, device="cuda")
    api.moe_grouped_gemm_fp8(codes, scales, off, w, ws, out, work)
    assert api.moe_get_device_status(work)[0] == BAD_OFFSETS


def test_grouped_product_not_finite_rows_stay_apart():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 256, generator=g).to(torch.bfloat16)
    x[2, 3], x[5, 200] = float("nan"), float("inf")
    codes, scales = _quantise(x)
    w, ws = _weights(g, 1, 128, 256)
    out = torch.empty(9, 128, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    api.moe_grouped_gemm_fp8(codes, scales, torch.tensor([0, 9], dtype=torch.int32, device="cuda"), w, ws, out, work)
    bad = torch.isnan(out).all(1).cpu()
    assert bad.tolist() == [i in (2, 5) for i in range(9)]
    assert torch.isfinite(out[~bad.cuda()]).all()


def test_grouped_product_many_groups_on_another_stream():
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    rows = sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    codes, scales = _quantise(torch.randn(rows, 64, generator=g).to(torch.bfloat16))
    w, ws = _weights(g, 1024, 32, 64)
    out = torch.empty(rows, 32, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(1024, rows, 32, 64), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = torch.from_numpy(off).cuda()
    s.wait_stream(torch.cuda.current_stream())
    api.moe_workspace_init(work, s)
    api.moe_grouped_gemm_fp8(codes, scales, o, w, ws, out, work, stream=s)
    assert api.moe_get_device_status(work, s) == (0, 0)
    ref, mag = _product_ref(codes, scales, off, w, ws, False)
    assert (np.abs(np32(out) - ref) <= _product_tol(ref, mag, 64)).all()


def _check_layer(cfg):
    p_cpu = make_layer(cfg, "cpu")
    p, h = to_dev(p_cpu), host_params(p_cpu)
    dy = make_dy(cfg, "cpu")
    layer = api.MoELayer(cfg, p, train=True)
    out = layer.forward(p["x"]).clone()
    gr = layer.backward(dy.cuda())
    torch.cuda.synchronize()
    assert layer.device_status()[0] == 0
    lg = O.gate_logits(h["x"], h["w_gate"])
    idx, g = O.route(lg, h.get("bias"), cfg.top_k, cfg.gate)
    keys = O.selection_keys(lg, h.get("bias"))
    tol = 2 * float(np.abs(np32(layer.buf["logits"]) - lg).max()) + 1e-6
    assert routing_agreement(keys, layer.buf["topk_idx"].cpu().numpy(), idx, tol).all()
    value = lambda key: O.fp8_tile_value(*O.fp8_tile_quantize(h[key]))  # noqa: E731
    w1, w3, w2 = value("w1"), value("w3"), value("w2")
    shared = (value("ws1"), value("ws3"), value("ws2")) if cfg.n_shared else None
    ref, saved = O.moe_forward_fp8b(h["x"], idx, g, w1, w3, w2, shared)
    assert rel(np32(out), ref) < BF16_TOL
    rg = O.moe_backward_fp8b(np32(dy), h["x"], lg, idx, g, h["w_gate"], w1, w3, w2, saved, cfg.gate, shared)
    for key in ("dx", "dw1", "dw3", "dw2", "dw_gate", "dg") + (("dws1", "dws3", "dws2") if cfg.n_shared else ()):
        assert rel(np32(gr[key]), rg[key]) < BF16_TOL, key
    used = np.unique(idx)
    for e in set(range(cfg.n_exp)) - set(used.tolist()):
        assert not gr["dw1"][e].any() and not gr["dw2"][e].any()
    # inference keeps no bf16 rows and gives the same bits, and so does a second run
    infer = api.MoELayer(cfg, p, train=False)
    assert torch.equal(infer.forward(p["x"]).view(torch.int16), out.view(torch.int16))
    assert torch.equal(layer.forward(p["x"]).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("name,tokens", [("tiny", None), ("small_softmax", None), ("small_sigmoid", None),
                                         ("small_fine", None), ("small_sigmoid", 1)])
def test_fp8b_layer_forward_backward(name, tokens):
    cfg = CONFIGS[name].replace(precision="fp8b")
    if tokens:
        cfg = cfg.replace(n_tok=tokens)
    _check_layer(cfg)


@pytest.mark.parametrize("tokens,d,f,e,k", [(1, 2048, 256, 4, 2), (3, 4096, 2048, 4, 1), (2, 7168, 320, 8, 4),
                                            (130, 2112, 192, 2, 1)])
def test_fp8b_layer_few_tokens(tokens, d, f, e, k):
    """Products of few tiles, split along the contraction."""
    _check_layer(MoEConfig("few", tokens, d, f, e, k, precision="fp8b"))


def test_permute_fp8b_rows():
    cfg = CONFIGS["small_fine"].replace(precision="fp8b")
    p = to_dev(make_layer(cfg, "cpu"))
    layer = api.MoELayer(cfg, p, train=True)
    layer.forward(p["x"])
    torch.cuda.synchronize()
    b = layer.buf
    for rows, codes, scales in (("x_perm", "xq_perm", "xs_perm"), (None, "xq_tok", "xs_tok")):
        x = b[rows] if rows else p["x"]
        rc, rs = O.fp8_rows_quantize(np32(x))
        np.testing.assert_array_equal(b[codes].cpu().numpy(), rc)
        np.testing.assert_array_equal(b[scales][:, :rs.shape[1]].cpu().numpy(), rs)


@pytest.mark.parametrize("mn", [False, True])
@pytest.mark.parametrize("sizes,n,k", [([700], 528, 400), ([300, 0, 900, 5], 256, 656), ([1, 40, 33], 2064, 144),
                                       ([512, 513], 272, 1296), ([1300, 900], 2320, 256)])
def test_grouped_product_tiles(sizes, n, k, mn):
    """Both tile widths, few and many rows a group, many column tiles."""
    g = torch.Generator().manual_seed(sum(sizes) + n + k)
    rows = sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    codes, scales = _quantise(torch.randn(rows, k, generator=g).to(torch.bfloat16))
    w, ws = _weights(g, len(sizes), *((k, n) if mn else (n, k)))
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(len(sizes), rows, n, k), dtype=torch.uint8,
                       device="cuda")
    api.moe_workspace_init(work)
    api.moe_grouped_gemm_fp8(codes, scales, torch.from_numpy(off).cuda(), w, ws, out, work, b_mn=mn)
    assert api.moe_get_device_status(work) == (0, 0)
    ref, mag = _product_ref(codes, scales, off, w, ws, mn)
    assert (np.abs(np32(out) - ref) <= _product_tol(ref, mag, k)).all()


def test_grouped_product_and_data_gradient_are_adjoint():
    """<a W^T, g> = <a, g W>: the forward and the data gradient of the same weights, on operands that
    are their own quantised values; each output element is off by the product's tolerance."""
    r = torch.Generator().manual_seed(5)
    rows, n, k = 200, 384, 640
    off = torch.tensor([0, 60, 200], dtype=torch.int32, device="cuda")
    w, ws = _weights(r, 2, n, k)
    work = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    val = lambda c, s, m: O.fp8_rows_dequantize(c.cpu().numpy(), s[:, :m // 128].cpu().numpy())  # noqa: E731
    a, sa = _quantise(torch.randn(rows, k, generator=r).to(torch.bfloat16))
    g, sg = _quantise(torch.randn(rows, n, generator=r).to(torch.bfloat16))
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    api.moe_grouped_gemm_fp8(a, sa, off, w, ws, y, work)
    api.moe_grouped_gemm_fp8(g, sg, off, w, ws, dx, work, b_mn=True)
    av, gv = val(a, sa, k), val(g, sg, n)
    left, right = np32(y).astype(np.float64) * gv, np32(dx).astype(np.float64) * av
    slack = lambda m: (2.0 ** -8 + 2.0 ** -12) * np.abs(m).sum()  # noqa: E731
    assert abs(left.sum() - right.sum()) <= slack(left) + slack(right)
    # and much closer, since the roundings are as often up as down: eight standard deviations
    dev = 2.0 ** -8 / np.sqrt(3) * np.sqrt((left ** 2).sum() + (right ** 2).sum())
    assert abs(left.sum() - right.sum()) <= 8 * dev + 2.0 ** -12 * (np.abs(left).sum() + np.abs(right).sum())
