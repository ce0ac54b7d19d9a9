"""Oracle of the FP8 layer with one fp32 scale per block of 128, of the layer
norm and of the counter-based dropout: numpy, 64 bits unless a value is stored
in fewer.

FP8 ("LLM Infrastructure Engineering 08: MoE Training Engineering" §13.6):
activations have one scale per 128 consecutive elements of a row, weights one
per 128 x 128 tile.  A row block's scale is the fp32 product amax * (1 / 448) (1
for an all-zero block), a weight tile's amax / 448; code = E4M3(x / scale).  Products are exact sums of the values the codes stand for.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import router_logit_grad
from .mxfp8 import bf16_round, e4m3_decode, e4m3_encode

BLOCK = 128


def fp8_rows_quantize(x: np.ndarray):
    """x [rows, cols] -> codes uint8 [rows, cols], scales fp32 [rows, ceil(cols / 128)]."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.ones((rows, nb), np.float32)
    for b in range(nb):
        blk = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        amax = np.abs(blk).max(axis=1).astype(np.float32)
        s = (amax * (np.float32(1.0) / np.float32(448.0))).astype(np.float32)
        scales[:, b] = np.where(s > 0, s, np.float32(1.0))
        codes[:, b * BLOCK:(b + 1) * BLOCK] = e4m3_encode(blk / scales[:, b:b + 1].astype(np.float64))
    return codes, scales


def fp8_rows_dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    s = np.repeat(scales.astype(np.float64), BLOCK, axis=1)[:, :codes.shape[1]]
    return e4m3_decode(codes) * s


def fp8_rows_value(x: np.ndarray) -> np.ndarray:
    """What the quantised rows of x stand for, in 64 bits."""
    return fp8_rows_dequantize(*fp8_rows_quantize(x))


def fp8_tile_value(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What E4M3 codes [..., rows, cols] with 128 x 128 tile scales stand for, in 64 bits."""
    r, c = codes.shape[-2:]
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=-2), BLOCK, axis=-1)[..., :r, :c]
    return e4m3_decode(codes) * s


def _sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def swiglu_expert_fp8b(x, w1, w3, w2):
    """One expert on values x (already quantised): y, a1, a3, h."""
    a1, a3 = x @ w1.T, x @ w3.T
    h = a1 * _sigmoid(a1) * a3
    return fp8_rows_value(h) @ w2.T, a1, a3, h


def moe_forward_fp8b(x, idx, g, w1, w3, w2, shared=None):
    """Forward on weight values w1, w3 [E,F,D], w2 [E,D,F]; returns out and what the backward needs."""
    n, d = x.shape
    xq = fp8_rows_value(x)
    out = np.zeros((n, d))
    saved = {"experts": {}, "shared": None}
    for e in range(w1.shape[0]):
        tok, kk = np.nonzero(idx == e)
        if tok.size:
            y, a1, a3, h = swiglu_expert_fp8b(xq[tok], w1[e], w3[e], w2[e])
            saved["experts"][e] = (tok, kk, y, a1, a3, h)
            np.add.at(out, tok, y * g[tok, kk].astype(np.float64)[:, None])
    if shared is not None:
        y, a1, a3, h = swiglu_expert_fp8b(xq, *shared)
        saved["shared"] = (a1, a3, h)
        out = out + y
    return out, saved


def moe_backward_fp8b(dy, x, logits, idx, g, w_gate, w1, w3, w2, saved, gate, shared=None):
    """Data gradients on FP8 operands quantised from the stored bf16 tensors, weight gradients from those tensors."""
    n, d = x.shape
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    dx = np.zeros((n, d))
    grads = {"dw1": np.zeros(w1.shape), "dw3": np.zeros(w3.shape), "dw2": np.zeros(w2.shape)}
    dg = np.zeros(idx.shape)
    store = lambda v: bf16_round(v.astype(np.float32)).astype(np.float64)  # noqa: E731

    def expert(dyw, xe, a1, a3, h, v1, v3, v2):
        dyw, a1, a3, h = store(dyw), store(a1), store(a3), store(h)
        dh = fp8_rows_value(dyw) @ v2
        s = _sigmoid(a1)
        da1, da3 = store(dh * a3 * s * (1.0 + a1 * (1.0 - s))), store(dh * a1 * s)
        gx = fp8_rows_value(da1) @ v1 + fp8_rows_value(da3) @ v3
        return da1.T @ xe, da3.T @ xe, dyw.T @ h, gx

    for e, (tok, kk, y, a1, a3, h) in saved["experts"].items():
        dg[tok, kk] = (dy[tok] * store(y)).sum(axis=1)
        r = expert(dy[tok] * g[tok, kk].astype(np.float64)[:, None], x[tok], a1, a3, h, w1[e], w3[e], w2[e])
        grads["dw1"][e], grads["dw3"][e], grads["dw2"][e] = r[:3]
        np.add.at(dx, tok, store(r[3]))
    if shared is not None:
        r = expert(dy, x, *saved["shared"], *shared)
        grads.update(dws1=r[0], dws3=r[1], dws2=r[2])
        dx = dx + store(r[3])
    dl = router_logit_grad(dg, g, logits, idx, gate, np.float64)
    grads.update(dx=dx + dl @ w_gate.astype(np.float64), dw_gate=dl.T @ x, dg=dg)
    return grads


def layernorm(x, gamma, beta, eps):
    """y, mean, rstd of the rows of x in 64 bits."""
    x = x.astype(np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(x.var(axis=1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + (0.0 if beta is None else beta), mean, rstd


def layernorm_backward(dy, x, gamma, eps, dres=None):
    """dx, dgamma, dbeta in 64 bits."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    _, mean, rstd = layernorm(x, gamma, None, eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    return dx + (0.0 if dres is None else dres.astype(np.float64)), (dy * xhat).sum(0), dy.sum(0)


def philox_words(seed: int, counter: int) -> list[int]:
    """The four words of one 64-bit counter (upper half zero): Philox-4x32 with
    ten rounds, J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
    numbers: as easy as 1, 2, 3" (2011), in Python integers."""
    m = 0xFFFFFFFF
    c = [counter & m, (counter >> 32) & m, 0, 0]
    k = [seed & m, (seed >> 32) & m]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def dropout_keep(seed: int, offset: int, n: int, p: float) -> np.ndarray:
    """Which of n elements stay."""
    low = (1 << 64) - 1
    words = [w for i in range(-(-n // 4)) for w in philox_words(seed & low, (offset + i) & low)]
    return np.array(words[:n], dtype=np.uint64) >= np.uint64(min(int(np.floor(p * 2.0 ** 32 + 0.5)), 0xFFFFFFFF))
