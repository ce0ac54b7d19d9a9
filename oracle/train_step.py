"""Oracle of a training step's operators beside the layer: the balance loss over
ragged sequences with the z-loss, the dense router gradient, and the backward from
activations kept in 8 bits.  64 bits throughout, a loop per sequence or expert.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np

from .mxfp8 import e4m3_decode

__all__ = ["balance_loss", "router_backward", "kept_values", "swiglu_backward_kept", "wgrad_kept"]


def _sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def gate_rows(l, gate):
    """The gate's distribution of every row and its slopes by their own logits.  Normalised sigmoids keep their ratios
    however low a row lies: their common factor e^m, m the largest logit where that is below zero, is left out."""
    m = l.max(axis=-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    if gate == "softmax":
        w = s = np.exp(l - m)
    else:
        s = np.exp(np.minimum(l, 0.0) - np.minimum(m, 0.0)) * _sigmoid(np.abs(l))
        w = s * _sigmoid(-l)
    tot = s.sum(axis=-1, keepdims=True)
    tot = np.where(tot > 0, tot, 1.0)
    return s / tot, w / tot


def balance_loss(logits, idx, seq_offsets, gate, coef, z_coef, f=None):
    """``coef E / S' sum_s sum_i f_si mean_t q_ti`` and ``z_coef / T sum_t lse_t^2`` over the sequences
    ``[o_s, o_{s+1})``, their gradient [N, E] and the counts [S, E].  ``f`` (optional, [S, E]) holds the fractions
    fixed at given values instead of counts / T_s (for differences)."""
    lg = np.asarray(logits, dtype=np.float64)
    n, e = lg.shape
    s_all = len(seq_offsets) - 1
    spans = [(int(a), int(b)) for a, b in zip(seq_offsets[:-1], seq_offsets[1:])]
    full = sum(b > a for a, b in spans)
    used = sum(b - a for a, b in spans)
    counts = np.zeros((s_all, e), np.int64)
    grad = np.zeros((n, e))
    balance = square = 0.0
    for s, (a, b) in enumerate(spans):
        if b <= a:
            continue
        counts[s] = np.bincount(np.asarray(idx[a:b]).ravel(), minlength=e)
        fs = counts[s] / (b - a) if f is None else f[s]
        l = lg[a:b]
        m = l.max(axis=1, keepdims=True)
        live = np.isfinite(m[:, 0])
        m = np.where(np.isfinite(m), m, 0.0)
        ex = np.exp(l - m)
        tot = np.where(live, ex.sum(axis=1), 1.0)[:, None]
        p = ex / tot
        lse = np.where(live, m[:, 0] + np.log(tot[:, 0]), 0.0)
        q, dq = gate_rows(l, gate)
        inner = q @ fs
        balance += coef * e / full * inner.mean()
        square += z_coef / used * (lse ** 2).sum()
        grad[a:b] = (coef * e / full / (b - a) * dq * (fs[None] - inner[:, None])
                     + 2 * z_coef / used * lse[:, None] * p)
    return counts, np.array([balance, square]), grad


def router_backward(dlogits, x, w_gate, dx_in, dw_in):
    """``dx_in + dlogits W_g`` and ``dw_in + dlogits^T x``."""
    dl = np.asarray(dlogits, dtype=np.float64)
    return dx_in + dl @ np.asarray(w_gate, np.float64), dw_in + dl.T @ np.asarray(x, np.float64)


def kept_values(codes, scales):
    """Values of kept rows: codes [rows, cols], scale bytes [cols / 32, ld >= rows]."""
    rows, cols = codes.shape
    s = np.exp2(np.asarray(scales)[:, :rows].astype(np.float64) - 127)
    return e4m3_decode(codes) * np.repeat(s.T, 32, axis=1)[:, :cols]


def swiglu_backward_kept(dy, offsets, w2, row_w, a1, a3):
    """da1, da3, the weighted h and dg for values a1, a3 of the kept rows; rows of no group stay NaN."""
    rows, f = a1.shape
    da1, da3, h = (np.full((rows, f), np.nan) for _ in range(3))
    dg = np.full(rows, np.nan)
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        dh = np.asarray(dy[r], np.float64) @ np.asarray(w2[e], np.float64)
        s = _sigmoid(a1[r])
        g = np.asarray(row_w[r], np.float64)[:, None]
        da1[r] = g * dh * a3[r] * s * (1.0 + a1[r] * (1.0 - s))
        da3[r] = g * dh * a1[r] * s
        h[r] = g * a1[r] * s * a3[r]
        dg[r] = (dh * a1[r] * s * a3[r]).sum(axis=1)
    return da1, da3, h, dg


def wgrad_kept(dy, x, offsets, row_map, row_div):
    """Per group the sum over its rows of dy[r]^T x[row_map[r] // row_div]."""
    out = np.zeros((len(offsets) - 1, dy.shape[1], x.shape[1]))
    src = np.asarray(row_map, np.int64) // row_div
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        out[e] = np.asarray(dy[r], np.float64).T @ x[src[r]]
    return out
