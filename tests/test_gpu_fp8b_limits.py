"""GPU parity of the FP8 blocks of 128 where their numbers end: every border
between two codes under every mantissa of a block's scale, blocks of h near the
end of fp32's range, and offsets that decrease."""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import BF16_TOL, np32, rel
from ragged_grouped_gemm_gb300 import api
from ragged_grouped_gemm_gb300.inputs import MoEConfig

pytestmark = pytest.mark.gpu
BAD_OFFSETS = 4


def _quantise(x):
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[0], api.fp8_scale_ld(x.shape[1]), device="cuda")
    api.moe_quantize_fp8_rows(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("exponent", [0, 15, -30, -66, -104, -126, 120])
def test_quantise_rows_every_mantissa_of_the_scale(exponent):
    """A block's largest magnitude takes all 128 bf16 mantissas of a binade, so its scale has every
    mantissa it can have; the others run through every bf16 magnitude down to amax / 2^21, past the
    smallest code (2^-9 of a scale that is amax / 448).  Whether a quotient lies just below
    or above a power of two, where the codes' spacing changes, depends on the scale's mantissa."""
    blocks = []
    for m in range(128):
        top = ((exponent + 127) << 7) + m                              # bf16 bits of amax
        bits = torch.arange(max(top - 21 * 128, 0), top + 1, dtype=torch.int32)
        v = (bits << 16).view(torch.float32)
        v = torch.cat([v, -v])
        v = torch.nn.functional.pad(v, (0, -v.numel() % 127)).view(-1, 127)
        amax = torch.tensor([top << 16], dtype=torch.int32).view(torch.float32)
        blocks.append(torch.cat([amax.expand(v.shape[0], 1), v], 1))
    x = torch.cat(blocks).to(torch.bfloat16)
    codes, scales = _quantise(x)
    rc, rs = O.fp8_rows_quantize(x.float().numpy())
    np.testing.assert_array_equal(scales[:, :1].cpu().numpy().view(np.uint32), rs.view(np.uint32))
    wrong = codes.cpu().numpy() != rc
    r, c = np.nonzero(wrong)
    assert not wrong.any(), (int(wrong.sum()), [(float(x[i, 0]), float(x[i, j]), int(codes[i, j]), int(rc[i, j]))
                                                for i, j in zip(r[:4], c[:4])])


def _tiles(g, e, r, c):
    w = (torch.randn(e, r, c, generator=g) * 0.05).to(torch.bfloat16).cuda()
    q = api.quantize_weights_fp8_tile({"w1": w})
    return q["w1"], q["w1_scale"]


@pytest.mark.parametrize("mn", [False, True])
@pytest.mark.parametrize("n,k", [(144, 128), (400, 1168), (144, 2048), (1040, 4112)])
@pytest.mark.parametrize("off", [[0, 300, 0, 300], [0, 300, 299, 300], [300, 0, 0, 300], [0, 10, 5, 5], [0, 400, 20, 300]])
def test_product_descending_offsets_are_flagged_and_write_nothing(off, n, k, mn):
    """In both the split (k from 2048) and the plain launch, whatever number of tiles they give."""
    g = torch.Generator().manual_seed(n + k)
    codes, scales = _quantise(torch.randn(300, k, generator=g).to(torch.bfloat16))
    w, ws = _tiles(g, 3, *((k, n) if mn else (n, k)))
    out = torch.full((300, n), 7.0, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(api.moe_grouped_gemm_fp8_workspace_size(3, 300, n, k), dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(work)
    api.moe_grouped_gemm_fp8(codes, scales, torch.tensor(off, dtype=torch.int32, device="cuda"), w, ws, out, work,
                             b_mn=mn)
    assert api.moe_get_device_status(work)[0] == BAD_OFFSETS
    assert (out == 7.0).all()
    # the same workspace and buffers go on with offsets that ascend
    api.moe_workspace_init(work)
    api.moe_grouped_gemm_fp8(codes, scales, torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda"), w, ws,
                             out, work, b_mn=mn)
    assert api.moe_get_device_status(work) == (0, 0)
    assert (out != 7.0).any(1).all()


def test_layer_products_descending_offsets_are_flagged():
    cfg = MoEConfig("descend", 64, 256, 192, 4, 2, precision="fp8b")
    g = torch.Generator().manual_seed(2)
    desc = api.make_desc(cfg)
    ws = torch.empty(api.moe_workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    codes, scales = _quantise(torch.randn(128, 256, generator=g).to(torch.bfloat16))
    wq = {}
    for key, r, c in (("w1", 192, 256), ("w3", 192, 256), ("w2", 256, 192)):
        wq[key], wq[key + "_scale"] = _tiles(g, 4, r, c)
    y = torch.full((128, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 128, 0, 128, 128], dtype=torch.int32, device="cuda")
    api.moe_grouped_ffn_fp8b(desc, codes, scales, off, None, None, wq, {}, y, None, ws)
    assert api.moe_get_device_status(ws)[0] == BAD_OFFSETS
    assert (y == 7.0).all()


@pytest.mark.parametrize("down", [0, -90, -113, -118])
@pytest.mark.parametrize("sizes,d,f", [([40, 0, 90], 256, 192), ([1, 2], 2048, 128)])
def test_layer_products_of_small_h(sizes, d, f, down):
    """h = silu(a1) a3 with a3 scaled down by 2^down and w2 up by as much: the largest magnitude of a
    block of h is then about 2^down, 2^-118 below 448e-37, and y stays of order one.  The scale
    products of a3 are about 2^-20 of it; the smallest keep 2^-149 / 2^-138 = 2^-11 of their
    value, half of that off (2^-12), a part of the tolerance of 5e-3."""
    g = torch.Generator().manual_seed(d - down)
    rows, e = sum(sizes), len(sizes)
    cfg = MoEConfig("small h", rows, d, f, e, 1, precision="fp8b")
    desc = api.make_desc(cfg)
    ws = torch.empty(api.moe_workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    codes, scales = _quantise(torch.randn(rows, d, generator=g).to(torch.bfloat16))
    wq = {}
    for key, r, c in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
        wq[key], wq[key + "_scale"] = _tiles(g, e, r, c)
    wq["w3_scale"] *= 2.0 ** down
    wq["w2_scale"] *= 2.0 ** -down
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    api.moe_grouped_ffn_fp8b(desc, codes, scales, torch.from_numpy(off).cuda(), None, None, wq, {}, y, None, ws)
    assert api.moe_get_device_status(ws) == (0, 0)
    x = O.fp8_rows_dequantize(codes.cpu().numpy(), scales[:, :-(-d // 128)].cpu().numpy())
    v = {k: O.fp8_tile_value(wq[k].cpu().numpy(), wq[k + "_scale"].cpu().numpy()) for k in ("w1", "w3", "w2")}
    want = np.zeros((rows, d))
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo < hi:
            want[lo:hi] = O.swiglu_expert_fp8b(x[lo:hi], v["w1"][i], v["w3"][i], v["w2"][i])[0]
    assert rel(np32(y), want) < BF16_TOL


def test_layer_rounds_its_expert_outputs_and_their_sum_and_nothing_else():
    """Against the formula with bf16 expert outputs the layer's output is off by what moves a value over
    a border: fp32 sums of 2048 products, about 2^-21 of their magnitude, change a share of 2^-13
    of the bf16 roundings by a step of 2^-8 (2^-14 in the norm), and a share of 2^-17 of h's codes (128
    a binade pair of 2^-4) by 2^-3, which is 2^-11.5 of the norm of h and so of y.  2^-10 in all, a third of the 2.7e-3
    that leaving out the first rounding makes.  A second run gives the same bits."""
    cfg = MoEConfig("rounds", 96, 2048, 512, 8, 4, precision="fp8b")
    g = torch.Generator().manual_seed(11)
    x = torch.randn(96, 2048, generator=g).to(torch.bfloat16)
    idx = torch.stack([torch.randperm(8, generator=g)[:4] for _ in range(96)]).to(torch.int32)
    w = torch.softmax(torch.randn(96, 4, generator=g), 1)
    off = np.concatenate([[0], np.cumsum(np.bincount(idx.numpy().ravel(), minlength=8))]).astype(np.int32)
    desc = api.make_desc(cfg)
    ws = torch.empty(api.moe_workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    api.moe_workspace_init(ws)
    wq = {}
    for key, r, c in (("w1", 512, 2048), ("w3", 512, 2048), ("w2", 2048, 512)):
        wq[key], wq[key + "_scale"] = _tiles(g, 8, r, c)
    rows, copies = (torch.empty(384, dtype=torch.int32, device="cuda") for _ in range(2))
    xq = torch.empty(384, 2048, dtype=torch.uint8, device="cuda")
    xs = torch.empty(384, api.fp8_scale_ld(2048), device="cuda")
    y = torch.empty(384, 2048, dtype=torch.bfloat16, device="cuda")
    outs = []
    for _ in range(2):
        out = torch.empty(96, 2048, dtype=torch.bfloat16, device="cuda")
        o = torch.from_numpy(off).cuda()
        api.moe_permute_fp8b(desc, x.cuda(), idx.cuda(), o, rows, copies, None, xq, xs, None, None, ws)
        api.moe_grouped_ffn_fp8b(desc, xq, xs, o, None, None, wq, {}, y, None, ws)
        api.moe_combine(desc, y, rows, w.cuda(), None, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    v = {k: O.fp8_tile_value(wq[k].cpu().numpy(), wq[k + "_scale"].cpu().numpy()) for k in ("w1", "w3", "w2")}
    xv, once, twice = O.fp8_rows_value(x.float().numpy()), np.zeros((96, 2048)), np.zeros((96, 2048))
    for e in range(8):
        tok, kk = np.nonzero(idx.numpy() == e)
        ye = O.swiglu_expert_fp8b(xv[tok], v["w1"][e], v["w3"][e], v["w2"][e])[0]
        gw = w.numpy()[tok, kk].astype(np.float64)[:, None]
        np.add.at(once, tok, ye * gw)
        np.add.at(twice, tok, O.bf16_round(ye.astype(np.float32)).astype(np.float64) * gw)
    stored = O.bf16_round(twice.astype(np.float32))
    assert rel(np32(outs[0]), stored) < 2.0 ** -10
    assert rel(np32(outs[0]), once) < (2.0 ** -8 / np.sqrt(3)) * np.sqrt(2)    # two evenly spread roundings at most
