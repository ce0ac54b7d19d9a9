"""Python binding of libmoe: one function per C entry point, same names.

Each function only marshals arguments (checks device, dtype, contiguity and
shape; passes ``data_ptr()`` and the current CUDA stream) and raises
:class:`MoEError` on a non-OK status.  All computation happens in the CUDA
kernels of libmoe.so.  :class:`MoELayer` owns the buffers of one layer and
calls the entry points in forward/backward order.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .inputs import MoEConfig

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        lib = _lib.load()
        super().__init__(f"{fn}: {lib.moe_status_string(code).decode()} (status {code})")
        self.code = code


def _check(fn: str, code: int):
    if code != 0:
        raise MoEError(fn, code)


def _p(t: torch.Tensor | None, dtype=None, shape=None, name="tensor"):
    if t is None:
        return None
    if (t.is_cuda and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)
            and t.is_contiguous()):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()   # a shape given as another kind of sequence


# The handle of the current stream without building a Stream object for it,
# which took 3 of the 11 us that one norm's enqueue did.  Neither looks whether CUDA is
# initialised: every call passes a CUDA tensor first.  Without them, the public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _s(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def make_desc(cfg: MoEConfig) -> _lib.MoeDesc:
    return _lib.MoeDesc(cfg.n_tok, cfg.d_model, cfg.d_ff, cfg.n_exp, cfg.top_k,
                        1 if cfg.gate == "sigmoid" else 0, 1 if cfg.use_bias else 0,
                        cfg.n_shared, cfg.d_ff_shared if cfg.n_shared else 0,
                        {"bf16": 0, "mxfp8": 1, "fp8w": 2, "fp8b": 4}[cfg.precision])


# --------------------------------------------------------------- entry points
def moe_workspace_size(desc: _lib.MoeDesc) -> tuple[int, int]:
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check("moe_workspace_size", _lib.load().moe_workspace_size(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check("moe_workspace_init", _lib.load().moe_workspace_init(_p(ws, name="ws"), ws.numel() * ws.element_size(),
                                                                _s(stream)))


def moe_get_device_status(ws: torch.Tensor, stream=None) -> tuple[int, int]:
    out = (ctypes.c_int32 * 2)()
    _check("moe_get_device_status", _lib.load().moe_get_device_status(_p(ws, name="ws"), out, _s(stream)))
    return out[0], out[1]


def moe_route(desc, x, w_gate, bias, logits, topk_idx, topk_w, counts, offsets, ws, stream=None):
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    _check("moe_route", _lib.load().moe_route(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(w_gate, BF16, (e, d), "w_gate"),
        _p(bias, F32, (e,), "bias"), _p(logits, F32, (n, e), "logits"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(topk_w, F32, (n, k), "topk_w"), _p(counts, I32, (e,), "counts"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_route_from_logits(desc, logits, bias, topk_idx, topk_w, counts, offsets, ws, stream=None):
    n, e, k = desc.n_tok, desc.n_exp, desc.top_k
    _check("moe_route_from_logits", _lib.load().moe_route_from_logits(
        ctypes.byref(desc), _p(logits, F32, (n, e), "logits"), _p(bias, F32, (e,), "bias"),
        _p(topk_idx, I32, (n, k), "topk_idx"), _p(topk_w, F32, (n, k), "topk_w"), _p(counts, I32, (e,), "counts"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_route_permute(desc, x, w_gate, bias, logits, topk_idx, topk_w, counts, offsets, row_of_copy, copy_of_row,
                      x_perm, ws, stream=None):
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_route_permute", _lib.load().moe_route_permute(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(w_gate, BF16, (e, d), "w_gate"),
        _p(bias, F32, (e,), "bias"), _p(logits, F32, (n, e), "logits"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(topk_w, F32, (n, k), "topk_w"), _p(counts, I32, (e,), "counts"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(row_of_copy, I32, (r,), "row_of_copy"), _p(copy_of_row, I32, (r,), "copy_of_row"),
        _p(x_perm, BF16, (r, d), "x_perm"), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_permute(desc, x, topk_idx, offsets, row_of_copy, copy_of_row, x_perm, ws, stream=None):
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_permute", _lib.load().moe_permute(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(copy_of_row, I32, (r,), "copy_of_row"), _p(x_perm, BF16, (r, d), "x_perm"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_permute_noalloc(desc, x, topk_idx, offsets, row_of_copy, copy_of_row, x_perm, stream=None):
    """moe_permute for callers that cannot provide a workspace (see moe.h):
    the chunk tables live in a fixed device array inside the library."""
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_permute_noalloc", _lib.load().moe_permute_noalloc(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(copy_of_row, I32, (r,), "copy_of_row"), _p(x_perm, BF16, (r, d), "x_perm"), _s(stream)))


def moe_grouped_ffn(desc, x_perm, offsets, x, w1, w3, w2, ws1, ws3, ws2, a1, a3, h, a1s, a3s, hs, y_perm,
                    y_shared, ws, stream=None):
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs = n * k, desc.d_ff_shared
    sh = desc.n_shared
    w = _lib.MoeExpertWeights(_p(w1, BF16, (e, f, d), "w1"), _p(w3, BF16, (e, f, d), "w3"),
                              _p(w2, BF16, (e, d, f), "w2"),
                              _p(ws1, BF16, (fs, d), "ws1") if sh else None,
                              _p(ws3, BF16, (fs, d), "ws3") if sh else None,
                              _p(ws2, BF16, (d, fs), "ws2") if sh else None)
    sv = _lib.MoeFfnSaved(_p(a1, BF16, (r, f), "a1"), _p(a3, BF16, (r, f), "a3"), _p(h, BF16, (r, f), "h"),
                          _p(a1s, BF16, (n, fs), "a1s") if sh else None,
                          _p(a3s, BF16, (n, fs), "a3s") if sh else None,
                          _p(hs, BF16, (n, fs), "hs") if sh else None)
    _check("moe_grouped_ffn", _lib.load().moe_grouped_ffn(
        ctypes.byref(desc), _p(x_perm, BF16, (r, d), "x_perm"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(x, BF16, (n, d), "x") if sh else None, ctypes.byref(w), ctypes.byref(sv),
        _p(y_perm, BF16, (r, d), "y_perm"), _p(y_shared, BF16, (n, d), "y_shared") if sh else None,
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_permute_maps(desc, topk_idx, offsets, row_of_copy, copy_of_row, ws, stream=None):
    """The permutation maps of moe_permute without copying any row."""
    n, e, k = desc.n_tok, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_permute_maps", _lib.load().moe_permute_maps(
        ctypes.byref(desc), _p(topk_idx, I32, (n, k), "topk_idx"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(row_of_copy, I32, (r,), "row_of_copy"), _p(copy_of_row, I32, (r,), "copy_of_row"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_ffn_gather(desc, x, copy_of_row, offsets, w1, w3, w2, ws1, ws3, ws2, a1, a3, h, a1s, a3s, hs,
                           y_perm, y_shared, ws, stream=None):
    """moe_grouped_ffn reading GEMM1's rows from x through copy_of_row (TMA gathers)."""
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs = n * k, desc.d_ff_shared
    sh = desc.n_shared
    w = _lib.MoeExpertWeights(_p(w1, BF16, (e, f, d), "w1"), _p(w3, BF16, (e, f, d), "w3"),
                              _p(w2, BF16, (e, d, f), "w2"),
                              _p(ws1, BF16, (fs, d), "ws1") if sh else None,
                              _p(ws3, BF16, (fs, d), "ws3") if sh else None,
                              _p(ws2, BF16, (d, fs), "ws2") if sh else None)
    sv = _lib.MoeFfnSaved(_p(a1, BF16, (r, f), "a1"), _p(a3, BF16, (r, f), "a3"), _p(h, BF16, (r, f), "h"),
                          _p(a1s, BF16, (n, fs), "a1s") if sh else None,
                          _p(a3s, BF16, (n, fs), "a3s") if sh else None,
                          _p(hs, BF16, (n, fs), "hs") if sh else None)
    _check("moe_grouped_ffn_gather", _lib.load().moe_grouped_ffn_gather(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(copy_of_row, I32, (r,), "copy_of_row"),
        _p(offsets, I32, (e + 1,), "offsets"), ctypes.byref(w), ctypes.byref(sv),
        _p(y_perm, BF16, (r, d), "y_perm"), _p(y_shared, BF16, (n, d), "y_shared") if sh else None,
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_combine(desc, y_perm, row_of_copy, topk_w, y_shared, out, stream=None):
    n, d, k = desc.n_tok, desc.d_model, desc.top_k
    r = n * k
    _check("moe_combine", _lib.load().moe_combine(
        ctypes.byref(desc), _p(y_perm, BF16, (r, d), "y_perm"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(topk_w, F32, (n, k), "topk_w"), _p(y_shared, BF16, (n, d), "y_shared"), _p(out, BF16, (n, d), "out"),
        _s(stream)))


def _bwd_structs(desc, state: dict, grads: dict, need_x_perm: bool = True):
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs, sh = n * k, desc.d_ff_shared, desc.n_shared
    S = state
    st = _lib.MoeFwdState(
        _p(S["x"], BF16, (n, d), "x"),
        _p(S.get("x_perm"), BF16, (r, d), "x_perm") if (need_x_perm or S.get("x_perm") is not None) else None,
        _p(S["logits"], F32, (n, e), "logits"),
        _p(S["topk_idx"], I32, (n, k), "topk_idx"), _p(S["topk_w"], F32, (n, k), "topk_w"),
        _p(S["offsets"], I32, (e + 1,), "offsets"), _p(S["row_of_copy"], I32, (r,), "row_of_copy"),
        _p(S["copy_of_row"], I32, (r,), "copy_of_row"), _p(S["a1"], BF16, (r, f), "a1"), _p(S["a3"], BF16, (r, f), "a3"),
        _p(S["h"], BF16, (r, f), "h"), _p(S["y_perm"], BF16, (r, d), "y_perm"),
        _p(S.get("a1s"), BF16, (n, fs), "a1s") if sh else None, _p(S.get("a3s"), BF16, (n, fs), "a3s") if sh else None,
        _p(S.get("hs"), BF16, (n, fs), "hs") if sh else None,
        _p(S.get("offsets_full"), I32, (e + 1,), "offsets_full"),
        _p(S.get("copy_of_row_full"), I32, (r,), "copy_of_row_full"))
    return st, _grads_struct(desc, grads)


def _grads_struct(desc, grads: dict):
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    fs, sh, G = desc.d_ff_shared, desc.n_shared, grads
    return _lib.MoeGrads(
        _p(G["dx"], BF16, (n, d), "dx"), _p(G["dw_gate"], F32, (e, d), "dw_gate"), _p(G["dw1"], F32, (e, f, d), "dw1"),
        _p(G["dw3"], F32, (e, f, d), "dw3"), _p(G["dw2"], F32, (e, d, f), "dw2"),
        _p(G.get("dws1"), F32, (fs, d), "dws1") if sh else None, _p(G.get("dws3"), F32, (fs, d), "dws3") if sh else None,
        _p(G.get("dws2"), F32, (d, fs), "dws2") if sh else None,
        _p(G.get("dg"), F32, (n, k), "dg"), _p(G.get("dlogits"), F32, (n, k), "dlogits"))


def _weights_struct(desc, weights: dict):
    d, f, e = desc.d_model, desc.d_ff, desc.n_exp
    fs, sh = desc.d_ff_shared, desc.n_shared
    return _lib.MoeExpertWeights(_p(weights["w1"], BF16, (e, f, d), "w1"), _p(weights["w3"], BF16, (e, f, d), "w3"),
                                 _p(weights["w2"], BF16, (e, d, f), "w2"),
                                 _p(weights.get("ws1"), BF16, (fs, d), "ws1") if sh else None,
                                 _p(weights.get("ws3"), BF16, (fs, d), "ws3") if sh else None,
                                 _p(weights.get("ws2"), BF16, (d, fs), "ws2") if sh else None)


def moe_backward(desc, w_gate, weights: dict, state: dict, dy, grads: dict, ws, stream=None):
    """``weights``: w1, w3, w2 (+ ws1, ws3, ws2); ``state``: the fields of
    moe_fwd_state_t; ``grads``: the fields of moe_grads_t (dg, dlogits optional)."""
    n, d, e = desc.n_tok, desc.d_model, desc.n_exp
    w = _weights_struct(desc, weights)
    st, gr = _bwd_structs(desc, state, grads)
    _check("moe_backward", _lib.load().moe_backward(
        ctypes.byref(desc), _p(w_gate, BF16, (e, d), "w_gate"), ctypes.byref(w), ctypes.byref(st),
        _p(dy, BF16, (n, d), "dy"), ctypes.byref(gr), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_permute_capacity(desc, x, topk_idx, offsets, capacity_factor: float, row_of_copy_full, copy_of_row_full,
                         kept_offsets, row_of_copy, copy_of_row, x_perm, n_dropped, ws, stream=None):
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_permute_capacity", _lib.load().moe_permute_capacity(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(offsets, I32, (e + 1,), "offsets"), ctypes.c_double(capacity_factor),
        _p(row_of_copy_full, I32, (r,), "row_of_copy_full"), _p(copy_of_row_full, I32, (r,), "copy_of_row_full"),
        _p(kept_offsets, I32, (e + 1,), "kept_offsets"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(copy_of_row, I32, (r,), "copy_of_row"), _p(x_perm, BF16, (r, d), "x_perm"),
        _p(n_dropped, I32, (1,), "n_dropped"), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_aux_loss(desc, logits, counts, loss, dlogits_aux=None, ws=None, coef: float = 1.0, stream=None):
    """``loss``: fp32 device tensor of one element; ``dlogits_aux``: optional
    fp32 [N, E] receiving the loss's logit gradient."""
    n, e = desc.n_tok, desc.n_exp
    _check("moe_aux_loss", _lib.load().moe_aux_loss(
        ctypes.byref(desc), _p(logits, F32, (n, e), "logits"), _p(counts, I32, (e,), "counts"), ctypes.c_float(coef),
        _p(loss, F32, (1,), "loss"), _p(dlogits_aux, F32, (n, e), "dlogits_aux"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_monitor_stats(counts_hist, stats, stream=None):
    """``counts_hist``: int32 [H, E] device tensor (one routing histogram per
    step); ``stats``: fp32 device tensor [3] <- min load, entropy, cold experts."""
    h, e = counts_hist.shape
    _check("moe_monitor_stats", _lib.load().moe_monitor_stats(
        e, _p(counts_hist, I32, (h, e), "counts_hist"), h, _p(stats, F32, (3,), "stats"), _s(stream)))


# --------------------------------------------------------------- kernel timing
TIMING_KINDS = {"gate": 0, "ffn_fwd": 1, "dgrad": 2, "wgrad": 3}


def moe_timing_enable(capacity: int = 4096):
    """Start timing the library's grouped-GEMM launches with CUDA events
    (``capacity`` launches at most; earlier records are cleared)."""
    _check("moe_timing_enable", _lib.load().moe_timing_enable(capacity))


def moe_timing_read(kind: str) -> tuple[float, int, int]:
    """(total milliseconds, timed launches, untimed launches) of one kind of
    grouped GEMM since moe_timing_enable; waits for the recorded events."""
    ms, n, u = ctypes.c_double(), ctypes.c_int64(), ctypes.c_int64()
    _check("moe_timing_read", _lib.load().moe_timing_read(TIMING_KINDS[kind], ctypes.byref(ms), ctypes.byref(n),
                                                          ctypes.byref(u)))
    return ms.value, n.value, u.value


def moe_timing_disable():
    _check("moe_timing_disable", _lib.load().moe_timing_disable())


def moe_selftest_wait_timeout(ws, limit_ns: int, site: int, stream=None):
    """Run the library's bounded-wait self-test (see moe.h): a wait that
    nothing completes runs out after ``limit_ns`` and reports through the
    status words of ``ws``."""
    _check("moe_selftest_wait_timeout", _lib.load().moe_selftest_wait_timeout(
        _p(ws, name="ws"), ws.numel() * ws.element_size(), int(limit_ns), int(site), _s(stream)))


def moe_selftest_layernorm_timeout(desc, x, gamma, mean, rstd, row: int, limit_ns: int, ws, y=None, dy=None, dx=None,
                                   dgamma=None, dbeta=None, stream=None):
    """The layer norm (``y``) or its backward (``dy`` and its outputs) in which the
    wait for row ``row`` runs out after ``limit_ns`` (see moe.h)."""
    n, d = desc.n_tok, desc.d_model
    _check("moe_selftest_layernorm_timeout", _lib.load().moe_selftest_layernorm_timeout(
        ctypes.byref(desc), _p(dy, BF16, (n, d), "dy"), _p(x, None, (n, d), "x"), _stream_type(x, "x"),
        _p(gamma, F32, (d,), "gamma"), _p(y, BF16, (n, d), "y"), _p(mean, F32, (n,), "mean"),
        _p(rstd, F32, (n,), "rstd"), _p(dx, x.dtype, (n, d), "dx"), _p(dgamma, F32, (d,), "dgamma"),
        _p(dbeta, F32, (d,), "dbeta"), int(row), int(limit_ns), _p(ws, name="ws"), ws.numel() * ws.element_size(),
        _s(stream)))


def moe_update_bias(desc, counts, bias, gamma: float, mode: int = 0, stream=None):
    _check("moe_update_bias", _lib.load().moe_update_bias(
        ctypes.byref(desc), _p(counts, I32, (desc.n_exp,), "counts"), _p(bias, F32, (desc.n_exp,), "bias"),
        ctypes.c_float(gamma), mode, _s(stream)))


# --------------------------------------------------------------- MXFP8 forward
U8 = torch.uint8


def mx_scale_ld(rows: int) -> int:
    """Leading dimension of an MXFP8 scale array (rows rounded up to 16)."""
    return (rows + 15) // 16 * 16


def moe_quantize_mxfp8(src, codes, scales, stream=None):
    """src bf16 [G, rows, cols] (or [rows, cols]) -> codes uint8 (same shape),
    scales uint8 [G, cols/32, ld] (or [cols/32, ld]), ld = mx_scale_ld(rows)."""
    g, rows, cols = (1,) + tuple(src.shape) if src.dim() == 2 else tuple(src.shape)
    ld = scales.shape[-1]
    _check("moe_quantize_mxfp8", _lib.load().moe_quantize_mxfp8(
        _p(src, BF16, name="src"), g, rows, cols, _p(codes, U8, tuple(src.shape), "codes"),
        _p(scales, U8, (scales.shape if src.dim() == 3 else (cols // 32, ld)), "scales"), ld, _s(stream)))


def quantize_weights_mxfp8(p: dict, stream=None) -> dict:
    """MXFP8 copies (codes, scales) of the expert weights in ``p``."""
    out = {}
    for key in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        w = p.get(key)
        if w is None:
            continue
        codes = torch.empty(w.shape, dtype=U8, device=w.device)
        rows, cols = w.shape[-2], w.shape[-1]
        sshape = (w.shape[0], cols // 32, mx_scale_ld(rows)) if w.dim() == 3 else (cols // 32, mx_scale_ld(rows))
        scales = torch.zeros(sshape, dtype=U8, device=w.device)
        moe_quantize_mxfp8(w, codes, scales, stream)
        out[key], out[key + "_scale"] = codes, scales
    return out


def moe_quantize_mxfp8_t(src, codes, scales, stream=None):
    """src bf16 [G, rows, cols] (or [rows, cols]) quantised along rows and
    transposed: codes uint8 [G, cols, rows], scales uint8 [G, rows/32, ld]
    (ld = scales.shape[-1] >= cols, a multiple of 16)."""
    g, rows, cols = (1,) + tuple(src.shape) if src.dim() == 2 else tuple(src.shape)
    ld = scales.shape[-1]
    cshape = (cols, rows) if src.dim() == 2 else (g, cols, rows)
    sshape = (rows // 32, ld) if src.dim() == 2 else (g, rows // 32, ld)
    _check("moe_quantize_mxfp8_t", _lib.load().moe_quantize_mxfp8_t(
        _p(src, BF16, name="src"), g, rows, cols, _p(codes, U8, cshape, "codes"), _p(scales, U8, sshape, "scales"),
        ld, _s(stream)))


def quantize_weights_mxfp8_t(p: dict, stream=None) -> dict:
    """Transposed MXFP8 copies of the expert weights for the backward's data
    gradients (quantised along the other weight dimension)."""
    out = {}
    for key in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        w = p.get(key)
        if w is None:
            continue
        rows, cols = w.shape[-2], w.shape[-1]
        lead = (w.shape[0],) if w.dim() == 3 else ()
        codes = torch.empty(lead + (cols, rows), dtype=U8, device=w.device)
        scales = torch.zeros(lead + (rows // 32, mx_scale_ld(cols)), dtype=U8, device=w.device)
        moe_quantize_mxfp8_t(w, codes, scales, stream)
        out[key], out[key + "_scale"] = codes, scales
    return out


def moe_backward_mxfp8(desc, w_gate, wt: dict, state: dict, dy, grads: dict, ws, stream=None):
    """Backward of the MXFP8 layer.  ``wt``: output of
    :func:`quantize_weights_mxfp8_t`; ``state`` as for :func:`moe_backward`
    (x_perm not needed)."""
    n, d, e, sh = desc.n_tok, desc.d_model, desc.n_exp, desc.n_shared
    w = _lib.MoeExpertWeightsMx(*[_p(wt.get(key)) if (sh or not key.startswith("ws")) else None
                                  for key in ("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale",
                                              "ws1", "ws1_scale", "ws3", "ws3_scale", "ws2", "ws2_scale")])
    st, gr = _bwd_structs(desc, state, grads, need_x_perm=False)
    _check("moe_backward_mxfp8", _lib.load().moe_backward_mxfp8(
        ctypes.byref(desc), _p(w_gate, BF16, (e, d), "w_gate"), ctypes.byref(w), ctypes.byref(st),
        _p(dy, BF16, (n, d), "dy"), ctypes.byref(gr), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


# --------------------------------------------------------------- FP8 weights
def quantize_weights_fp8_tile(p: dict, stream=None) -> dict:
    """E4M3 codes with one fp32 scale per 128 x 128 tile of every expert
    weight in ``p`` (keys w1, w3, w2, ws1, ws3, ws2 and *_scale)."""
    out = {}
    for key in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        w = p.get(key)
        if w is None:
            continue
        g, rows, cols = (1,) + tuple(w.shape) if w.dim() == 2 else tuple(w.shape)
        codes = torch.empty(w.shape, dtype=U8, device=w.device)
        lead = (w.shape[0],) if w.dim() == 3 else ()
        scales = torch.empty(lead + ((rows + 127) // 128, (cols + 127) // 128), dtype=F32, device=w.device)
        _check("moe_quantize_fp8_tile", _lib.load().moe_quantize_fp8_tile(
            _p(w, BF16, name=key), g, rows, cols, _p(codes, U8, name=key + " codes"),
            _p(scales, F32, name=key + " scales"), _s(stream)))
        out[key], out[key + "_scale"] = codes, scales
    return out


def _mx_struct(desc, wq):
    sh = desc.n_shared
    return _lib.MoeExpertWeightsMx(*[_p(wq.get(key)) if (sh or not key.startswith("ws")) else None
                                     for key in ("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale",
                                                 "ws1", "ws1_scale", "ws3", "ws3_scale", "ws2", "ws2_scale")])


def moe_grouped_ffn_fp8w(desc, x_perm, offsets, x, wq: dict, saved: dict, y_perm, y_shared, ws, stream=None):
    """``wq``: output of :func:`quantize_weights_fp8_tile`; other arguments as
    :func:`moe_grouped_ffn` (``saved``: a1, a3, h, a1s, a3s, hs)."""
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r, sh = n * k, desc.n_shared
    w = _mx_struct(desc, wq)
    sv = _lib.MoeFfnSaved(*[_p(saved.get(key)) for key in ("a1", "a3", "h", "a1s", "a3s", "hs")])
    _check("moe_grouped_ffn_fp8w", _lib.load().moe_grouped_ffn_fp8w(
        ctypes.byref(desc), _p(x_perm, BF16, (r, d), "x_perm"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(x, BF16, (n, d), "x"), ctypes.byref(w), ctypes.byref(sv), _p(y_perm, BF16, (r, d), "y_perm"),
        _p(y_shared, BF16, (n, d), "y_shared") if sh else None, _p(ws, name="ws"), ws.numel() * ws.element_size(),
        _s(stream)))


def moe_backward_fp8w(desc, w_gate, wq: dict, state: dict, dy, grads: dict, ws, stream=None):
    n, d, e = desc.n_tok, desc.d_model, desc.n_exp
    w = _mx_struct(desc, wq)
    st, gr = _bwd_structs(desc, state, grads)
    _check("moe_backward_fp8w", _lib.load().moe_backward_fp8w(
        ctypes.byref(desc), _p(w_gate, BF16, (e, d), "w_gate"), ctypes.byref(w), ctypes.byref(st),
        _p(dy, BF16, (n, d), "dy"), ctypes.byref(gr), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_permute_mxfp8(desc, x, topk_idx, offsets, row_of_copy, copy_of_row, xq_perm, xs_perm, xq_tok, xs_tok, ws,
                      stream=None):
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r = n * k
    _check("moe_permute_mxfp8", _lib.load().moe_permute_mxfp8(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(copy_of_row, I32, (r,), "copy_of_row"), _p(xq_perm, U8, (r, d), "xq_perm"),
        _p(xs_perm, U8, (d // 32, mx_scale_ld(r)), "xs_perm"), _p(xq_tok, U8, (n, d), "xq_tok"),
        _p(xs_tok, U8, (d // 32, mx_scale_ld(n)), "xs_tok"), _p(ws, name="ws"), ws.numel() * ws.element_size(),
        _s(stream)))


def moe_grouped_ffn_mxfp8(desc, xq_perm, xs_perm, offsets, xq_tok, xs_tok, wq: dict, saved: dict, y_perm, y_shared,
                          ws, stream=None):
    """``wq``: output of :func:`quantize_weights_mxfp8`; ``saved``: optional bf16
    a1, a3, h, a1s, a3s, hs for a bf16 backward (missing keys = not saved)."""
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs, sh = n * k, desc.d_ff_shared, desc.n_shared
    w = _lib.MoeExpertWeightsMx(*[_p(wq.get(key)) if (sh or not key.startswith("ws")) else None
                                  for key in ("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale",
                                              "ws1", "ws1_scale", "ws3", "ws3_scale", "ws2", "ws2_scale")])
    sv = _lib.MoeFfnSaved(*[_p(saved.get(key)) for key in ("a1", "a3", "h", "a1s", "a3s", "hs")])
    _check("moe_grouped_ffn_mxfp8", _lib.load().moe_grouped_ffn_mxfp8(
        ctypes.byref(desc), _p(xq_perm, U8, (r, d), "xq_perm"), _p(xs_perm, U8, (d // 32, mx_scale_ld(r)), "xs_perm"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(xq_tok, U8, (n, d), "xq_tok") if sh else None,
        _p(xs_tok, U8, (d // 32, mx_scale_ld(n)), "xs_tok") if sh else None, ctypes.byref(w), ctypes.byref(sv),
        _p(y_perm, BF16, (r, d), "y_perm"), _p(y_shared, BF16, (n, d), "y_shared") if sh else None,
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


# --------------------------------------------------- FP8 with blocks of 128
def fp8_scale_ld(cols: int) -> int:
    """Floats per row of an activation's 1 x 128 block scales (MOE_FP8_SCALE_LD)."""
    return ((cols + 127) // 128 + 3) // 4 * 4


def moe_quantize_fp8_rows(src, codes, scales, stream=None):
    """src bf16 [rows, cols] -> codes uint8 [rows, cols], scales fp32 [rows, ld]
    (one per 128 columns; ld >= ceil(cols / 128), see :func:`fp8_scale_ld`)."""
    rows, cols = src.shape
    _check("moe_quantize_fp8_rows", _lib.load().moe_quantize_fp8_rows(
        _p(src, BF16, name="src"), rows, cols, _p(codes, U8, (rows, cols), "codes"),
        _p(scales, F32, (rows, scales.shape[-1]), "scales"), scales.shape[-1], _s(stream)))


def moe_grouped_gemm_fp8_workspace_size(n_groups: int, rows: int, n: int, k: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_grouped_gemm_fp8_workspace_size", _lib.load().moe_grouped_gemm_fp8_workspace_size(
        n_groups, rows, n, k, ctypes.byref(b)))
    return b.value


def moe_grouped_gemm_fp8(a, a_scale, offsets, b, b_scale, out, ws, b_mn: bool = False, stream=None):
    """out[r] = a[r] B_g^T for the rows of every group: a [rows, k] codes with
    a_scale [rows, ld]; b [G, n, k] codes (``b_mn``: [G, k, n]) with one scale
    per 128 x 128 tile; out bf16 [rows, n]."""
    if b.dim() != 3:
        raise ValueError(f"b must have three dimensions, got {tuple(b.shape)}")
    rows, k = a.shape
    g, n = b.shape[0], b.shape[2] if b_mn else b.shape[1]
    tiles = (g,) + tuple((v + 127) // 128 for v in b.shape[1:])
    _check("moe_grouped_gemm_fp8", _lib.load().moe_grouped_gemm_fp8(
        g, rows, n, k, _p(a, U8, name="a"), _p(a_scale, F32, (rows, a_scale.shape[-1]), "a_scale"),
        a_scale.shape[-1], _p(offsets, I32, (g + 1,), "offsets"), _p(b, U8, (g, k, n) if b_mn else (g, n, k), "b"),
        _p(b_scale, F32, tiles, "b_scale"), 1 if b_mn else 0, _p(out, BF16, (rows, n), "out"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_permute_fp8b(desc, x, topk_idx, offsets, row_of_copy, copy_of_row, x_perm, xq_perm, xs_perm, xq_tok, xs_tok,
                     ws, stream=None):
    """``x_perm`` (bf16 rows) and ``xq_tok``, ``xs_tok`` (token rows) may be None."""
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    r, ld = n * k, fp8_scale_ld(desc.d_model)
    _check("moe_permute_fp8b", _lib.load().moe_permute_fp8b(
        ctypes.byref(desc), _p(x, BF16, (n, d), "x"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(row_of_copy, I32, (r,), "row_of_copy"),
        _p(copy_of_row, I32, (r,), "copy_of_row"), _p(x_perm, BF16, (r, d), "x_perm"),
        _p(xq_perm, U8, (r, d), "xq_perm"), _p(xs_perm, F32, (r, ld), "xs_perm"), _p(xq_tok, U8, (n, d), "xq_tok"),
        _p(xs_tok, F32, (n, ld), "xs_tok"), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def _fp8_struct(desc, wq):
    d, f, e, fs = desc.d_model, desc.d_ff, desc.n_exp, desc.d_ff_shared
    shapes = {"w1": (e, f, d), "w3": (e, f, d), "w2": (e, d, f)}
    if desc.n_shared:
        shapes.update(ws1=(fs, d), ws3=(fs, d), ws2=(d, fs))
    ptr = []
    for key in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        shape = shapes.get(key)
        if shape is None:
            ptr += [None, None]
            continue
        tiles = shape[:-2] + tuple((v + 127) // 128 for v in shape[-2:])
        ptr += [_p(wq[key], U8, shape, key), _p(wq[key + "_scale"], F32, tiles, key + "_scale")]
    return _lib.MoeExpertWeightsMx(*ptr)


def moe_grouped_ffn_fp8b(desc, xq_perm, xs_perm, offsets, xq_tok, xs_tok, wq: dict, saved: dict, y_perm, y_shared,
                         ws, stream=None):
    """``wq``: output of :func:`quantize_weights_fp8_tile`; ``saved``: optional
    bf16 a1, a3, h, a1s, a3s, hs for the backward (missing keys = not saved)."""
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs, sh, ld = n * k, desc.d_ff_shared, desc.n_shared, fp8_scale_ld(desc.d_model)
    w = _fp8_struct(desc, wq)
    sv = _lib.MoeFfnSaved(*[_p(saved.get(key), BF16, (n, fs) if key.endswith("s") else (r, f), key)
                            for key in ("a1", "a3", "h", "a1s", "a3s", "hs")])
    _check("moe_grouped_ffn_fp8b", _lib.load().moe_grouped_ffn_fp8b(
        ctypes.byref(desc), _p(xq_perm, U8, (r, d), "xq_perm"), _p(xs_perm, F32, (r, ld), "xs_perm"),
        _p(offsets, I32, (e + 1,), "offsets"), _p(xq_tok, U8, (n, d), "xq_tok") if sh else None,
        _p(xs_tok, F32, (n, ld), "xs_tok") if sh else None, ctypes.byref(w), ctypes.byref(sv),
        _p(y_perm, BF16, (r, d), "y_perm"), _p(y_shared, BF16, (n, d), "y_shared") if sh else None,
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_backward_fp8b(desc, w_gate, wq: dict, state: dict, dy, grads: dict, ws, stream=None):
    n, d, e = desc.n_tok, desc.d_model, desc.n_exp
    w = _fp8_struct(desc, wq)
    st, gr = _bwd_structs(desc, state, grads)
    _check("moe_backward_fp8b", _lib.load().moe_backward_fp8b(
        ctypes.byref(desc), _p(w_gate, BF16, (e, d), "w_gate"), ctypes.byref(w), ctypes.byref(st),
        _p(dy, BF16, (n, d), "dy"), ctypes.byref(gr), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


# --------------------------------------------------------- the pre-norm block
def _stream_type(t, name: str) -> int:
    """0 for a bf16 residual stream, 1 for an fp32 one."""
    if t.dtype not in (BF16, F32):
        raise ValueError(f"{name} must be {BF16} or {F32}, got {t.dtype}")
    return int(t.dtype == F32)


def moe_layernorm(desc, x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """x [N, D] bf16 or fp32 -> y bf16; gamma, beta fp32 [D] (beta may be None);
    mean, rstd fp32 [N] for the backward (None in inference)."""
    n, d = desc.n_tok, desc.d_model
    _check("moe_layernorm", _lib.load().moe_layernorm(
        ctypes.byref(desc), _p(x, None, (n, d), "x"), _stream_type(x, "x"), _p(gamma, F32, (d,), "gamma"),
        _p(beta, F32, (d,), "beta"), float(eps), _p(y, BF16, (n, d), "y"), _p(mean, F32, (n,), "mean"),
        _p(rstd, F32, (n,), "rstd"), _s(stream)))


def moe_layernorm_backward(desc, dy, x, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream=None):
    """``dres`` (None: zero) is the gradient that reaches x past the norm and is
    added to dx; both have x's type.  ``dbeta`` may be None."""
    n, d = desc.n_tok, desc.d_model
    _check("moe_layernorm_backward", _lib.load().moe_layernorm_backward(
        ctypes.byref(desc), _p(dy, BF16, (n, d), "dy"), _p(x, None, (n, d), "x"), _stream_type(x, "x"),
        _p(gamma, F32, (d,), "gamma"), _p(mean, F32, (n,), "mean"), _p(rstd, F32, (n,), "rstd"),
        _p(dres, x.dtype, (n, d), "dres"), _p(dx, x.dtype, (n, d), "dx"), _p(dgamma, F32, (d,), "dgamma"),
        _p(dbeta, F32, (d,), "dbeta"), _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_combine_dropout(desc, y_perm, row_of_copy, topk_w, y_shared, resid, rng, p: float, out, stream=None):
    """moe_combine, dropout and the residual sum; ``resid`` (None: zero) and
    ``out`` bf16 or fp32; ``rng``: int64 device tensor [2] = seed, offset."""
    n, d, k = desc.n_tok, desc.d_model, desc.top_k
    _check("moe_combine_dropout", _lib.load().moe_combine_dropout(
        ctypes.byref(desc), _p(y_perm, BF16, (n * k, d), "y_perm"), _p(row_of_copy, I32, (n * k,), "row_of_copy"),
        _p(topk_w, F32, (n, k), "topk_w"), _p(y_shared, BF16, (n, d), "y_shared"),
        _p(resid, out.dtype, (n, d), "resid"), _stream_type(out, "out"), _p(rng, torch.int64, (2,), "rng"), float(p),
        _p(out, None, (n, d), "out"), _s(stream)))


def moe_dropout_backward(desc, dout, rng, p: float, dy, stream=None):
    """dy (bf16) = mask / (1 - p) * dout with the mask of moe_combine_dropout for the same ``rng``."""
    n, d = desc.n_tok, desc.d_model
    _check("moe_dropout_backward", _lib.load().moe_dropout_backward(
        ctypes.byref(desc), _p(dout, None, (n, d), "dout"), _stream_type(dout, "dout"),
        _p(rng, torch.int64, (2,), "rng"), float(p), _p(dy, BF16, (n, d), "dy"), _s(stream)))


# ------------------------------------------------------ balance over sequences
def moe_balance_loss(desc, logits, topk_idx, seq_offsets, counts, loss, dlogits=None, ws=None, coef: float = 1.0,
                     z_coef: float = 0.0, dloss=None, stream=None):
    """Balance loss over ragged sequences and the router's z-loss: ``seq_offsets``
    int32 [S + 1] (tokens of no sequence are padding); ``counts`` int32 [S, E],
    ``loss`` fp32 [2] = balance, z; ``dlogits`` fp32 [N, E] their gradient times
    ``dloss`` (one float on the device, None: 1)."""
    n, e, k = desc.n_tok, desc.n_exp, desc.top_k
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        raise ValueError(f"seq_offsets must have one dimension and two entries at least, got {tuple(seq_offsets.shape)}")
    s = seq_offsets.shape[0] - 1
    _check("moe_balance_loss", _lib.load().moe_balance_loss(
        ctypes.byref(desc), _p(logits, F32, (n, e), "logits"), _p(topk_idx, I32, (n, k), "topk_idx"),
        _p(seq_offsets, I32, (s + 1,), "seq_offsets"), s, float(coef), float(z_coef), _p(dloss, F32, (1,), "dloss"),
        _p(counts, I32, (s, e), "counts"), _p(loss, F32, (2,), "loss"), _p(dlogits, F32, (n, e), "dlogits"),
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_router_backward(desc, dlogits, x, w_gate, dx_in, dx, dw_in, dw_gate, ws, stream=None):
    """dx (bf16) = dx_in + dlogits W_g and dw_gate (fp32) = dw_in + dlogits^T x for
    a dense ``dlogits`` fp32 [N, E]; ``dx_in``, ``dw_in`` may be None or the outputs."""
    n, d, e = desc.n_tok, desc.d_model, desc.n_exp
    _check("moe_router_backward", _lib.load().moe_router_backward(
        ctypes.byref(desc), _p(dlogits, F32, (n, e), "dlogits"), _p(x, BF16, (n, d), "x"),
        _p(w_gate, BF16, (e, d), "w_gate"), _p(dx_in, BF16, (n, d), "dx_in"), _p(dx, BF16, (n, d), "dx"),
        _p(dw_in, F32, (e, d), "dw_in"), _p(dw_gate, F32, (e, d), "dw_gate"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


# ------------------------------------------------- 8-bit activation checkpoints
def moe_ckpt_workspace_size(desc) -> int:
    b = ctypes.c_size_t()
    _check("moe_ckpt_workspace_size", _lib.load().moe_ckpt_workspace_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def ckpt_buffers(desc, device="cuda") -> dict:
    """What one layer keeps for :func:`moe_backward_ckpt` in 8 bits: codes and
    scales of a1, a3 (a1s, a3s with a shared expert) and of the input x."""
    n, d, f = desc.n_tok, desc.d_model, desc.d_ff
    shapes = {"x": (n, d), "a1": (n * desc.top_k, f), "a3": (n * desc.top_k, f)}
    if desc.n_shared:
        shapes.update(a1s=(n, desc.d_ff_shared), a3s=(n, desc.d_ff_shared))
    out = {}
    for key, (rows, cols) in shapes.items():
        out[key] = torch.empty(rows, cols, dtype=U8, device=device)
        out[key + "_scale"] = torch.empty(cols // 32, mx_scale_ld(rows), dtype=U8, device=device)
    return out


def _ckpt_struct(desc, kept: dict):
    ptr = []
    for key in ("a1", "a3", "a1s", "a3s"):
        shared = key.endswith("s")
        if shared and not desc.n_shared:
            ptr += [None, None]
            continue
        rows, cols = (desc.n_tok, desc.d_ff_shared) if shared else (desc.n_tok * desc.top_k, desc.d_ff)
        ptr += [_p(kept[key], U8, (rows, cols), key),
                _p(kept[key + "_scale"], U8, (cols // 32, mx_scale_ld(rows)), key + "_scale")]
    return _lib.MoeCkpt(*ptr)


def moe_grouped_ffn_ckpt(desc, x_perm, offsets, x, weights: dict, kept: dict, y_perm, y_shared, ws, stream=None):
    """:func:`moe_grouped_ffn` that keeps a1 and a3 in 8 bits (``kept``:
    :func:`ckpt_buffers`) and no other activation."""
    n, d, f, e, k = desc.n_tok, desc.d_model, desc.d_ff, desc.n_exp, desc.top_k
    r, fs, sh = n * k, desc.d_ff_shared, desc.n_shared
    w = _weights_struct(desc, weights)
    _check("moe_grouped_ffn_ckpt", _lib.load().moe_grouped_ffn_ckpt(
        ctypes.byref(desc), _p(x_perm, BF16, (r, d), "x_perm"), _p(offsets, I32, (e + 1,), "offsets"),
        _p(x, BF16, (n, d), "x") if sh else None, ctypes.byref(w), ctypes.byref(_ckpt_struct(desc, kept)),
        _p(y_perm, BF16, (r, d), "y_perm"), _p(y_shared, BF16, (n, d), "y_shared") if sh else None,
        _p(ws, name="ws"), ws.numel() * ws.element_size(), _s(stream)))


def moe_backward_ckpt(desc, w_gate, weights: dict, state: dict, dy, grads: dict, ws, stream=None):
    """:func:`moe_backward` from 8-bit checkpoints.  ``state``: the codes and scales of
    :func:`ckpt_buffers` (x from :func:`moe_quantize_mxfp8`) and logits, topk_idx, topk_w, offsets,
    row_of_copy, copy_of_row of the forward."""
    n, d, e, k = desc.n_tok, desc.d_model, desc.n_exp, desc.top_k
    S = state
    st = _lib.MoeCkptState(
        _p(S["x"], U8, (n, d), "x"), _p(S["x_scale"], U8, (d // 32, mx_scale_ld(n)), "x_scale"),
        _p(S["logits"], F32, (n, e), "logits"), _p(S["topk_idx"], I32, (n, k), "topk_idx"),
        _p(S["topk_w"], F32, (n, k), "topk_w"), _p(S["offsets"], I32, (e + 1,), "offsets"),
        _p(S["row_of_copy"], I32, (n * k,), "row_of_copy"), _p(S["copy_of_row"], I32, (n * k,), "copy_of_row"),
        _ckpt_struct(desc, S))
    _check("moe_backward_ckpt", _lib.load().moe_backward_ckpt(
        ctypes.byref(desc), _p(w_gate, BF16, (e, d), "w_gate"), ctypes.byref(_weights_struct(desc, weights)),
        ctypes.byref(st), _p(dy, BF16, (n, d), "dy"), ctypes.byref(_grads_struct(desc, grads)), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_swiglu_backward_ckpt_workspace_size(n_groups: int, rows: int, d: int, f: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_swiglu_backward_ckpt_workspace_size", _lib.load().moe_swiglu_backward_ckpt_workspace_size(
        n_groups, rows, d, f, ctypes.byref(b)))
    return b.value


def moe_swiglu_backward_ckpt(dy, offsets, w2, row_w, a1, a1_scale, a3, a3_scale, da1, da3, h, dg, ws, stream=None):
    """The backward through w2 [G, d, f] and the SwiGLU from kept a1, a3 (codes uint8
    [rows, f], scales uint8 [f / 32, ld]) for dy bf16 [rows, d]: da1, da3 and the weighted h, bf16
    [rows, f], and dg fp32 [rows] (or None), the gradient of ``row_w`` (fp32 [rows], None: 1)."""
    if w2.dim() != 3 or a1_scale.dim() != 2:
        raise ValueError(f"w2 must have three dimensions and a1_scale two, got {tuple(w2.shape)}, "
                         f"{tuple(a1_scale.shape)}")
    g, d, f = w2.shape
    rows, ld = dy.shape[0], a1_scale.shape[-1]
    _check("moe_swiglu_backward_ckpt", _lib.load().moe_swiglu_backward_ckpt(
        g, rows, d, f, _p(dy, BF16, (rows, d), "dy"), _p(offsets, I32, (g + 1,), "offsets"),
        _p(w2, BF16, (g, d, f), "w2"), _p(row_w, F32, (rows,), "row_w"), _p(a1, U8, (rows, f), "a1"),
        _p(a1_scale, U8, (f // 32, ld), "a1_scale"), _p(a3, U8, (rows, f), "a3"),
        _p(a3_scale, U8, (f // 32, ld), "a3_scale"), ld, _p(da1, BF16, (rows, f), "da1"),
        _p(da3, BF16, (rows, f), "da3"), _p(h, BF16, (rows, f), "h"), _p(dg, F32, (rows,), "dg"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_wgrad_ckpt_workspace_size(n_groups: int, rows: int, m: int, k: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_grouped_wgrad_ckpt_workspace_size", _lib.load().moe_grouped_wgrad_ckpt_workspace_size(
        n_groups, rows, m, k, ctypes.byref(b)))
    return b.value


def moe_grouped_wgrad_ckpt(dy, x, x_scale, offsets, row_map, row_div: int, dw, ws, stream=None):
    """dw fp32 [G, m, k]: per group the sum over its rows of dy[r]^T x[row_map[r] // row_div] for dy
    bf16 [rows, m] and kept rows x (codes uint8 [x_rows, k], scales uint8 [k / 32, ld]).  ``row_map``
    None (with row_div 1): row r."""
    if dw.dim() != 3 or x_scale.dim() != 2:
        raise ValueError(f"dw must have three dimensions and x_scale two, got {tuple(dw.shape)}, "
                         f"{tuple(x_scale.shape)}")
    g, m, k = dw.shape
    rows, x_rows, ld = dy.shape[0], x.shape[0], x_scale.shape[-1]
    _check("moe_grouped_wgrad_ckpt", _lib.load().moe_grouped_wgrad_ckpt(
        g, rows, m, k, _p(dy, BF16, (rows, m), "dy"), _p(x, U8, (x_rows, k), "x"),
        _p(x_scale, U8, (k // 32, ld), "x_scale"), x_rows, ld, _p(row_map, I32, (rows,), "row_map"), int(row_div),
        _p(offsets, I32, (g + 1,), "offsets"), _p(dw, F32, (g, m, k), "dw"), _p(ws, name="ws"),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_dequantize_mxfp8(codes, scales, out, stream=None):
    """The values of MXFP8 rows (codes uint8 [rows, cols], scales uint8 [cols / 32, ld]) in bf16."""
    rows, cols = codes.shape
    _check("moe_dequantize_mxfp8", _lib.load().moe_dequantize_mxfp8(
        _p(codes, U8, name="codes"), _p(scales, U8, (cols // 32, scales.shape[-1]), "scales"), rows, cols,
        scales.shape[-1], _p(out, BF16, (rows, cols), "out"), _s(stream)))


# --------------------------------------------------------------- layer runner
class MoELayer:
    """Buffers of one layer plus the forward / backward call sequences.

    ``params``: x-independent tensors from :func:`inputs.make_layer` on the GPU
    (w_gate, w1, w3, w2, bias, and ws1, ws3, ws2 with a shared expert).

    ``checkpoint``: the forward keeps a1, a3 and x for the backward in 8 bits
    (``ckpt``, about 2 R F + N D bytes) instead of 6 R F + 4 R D bytes of bf16
    activations, and x itself is not read again.  ``share``: another
    checkpointing layer of the same shapes, whose workspace and buffers in
    passing (permuted rows, expert outputs) this layer uses as well; layers that
    share run one after another on one stream, and a layer's ``experts`` and its
    combine come one after the other.
    """

    def __init__(self, cfg: MoEConfig, params: dict, train: bool = True, device="cuda", gather: bool = False,
                 fused_dispatch: bool = True, checkpoint: bool = False, share: "MoELayer | None" = None):
        if checkpoint and (not train or cfg.precision != "bf16" or cfg.capacity_factor > 0):
            raise ValueError("8-bit checkpoints are kept by bf16 layers in training, without a capacity")
        if share is not None and not (checkpoint and share.ckpt is not None
                                      and bytes(make_desc(cfg)) == bytes(share.desc)):
            raise ValueError("a layer shares buffers with a checkpointing layer of the same shapes only")
        self.cfg = cfg
        self.desc = make_desc(cfg)
        self.p = params
        self.train = train
        n, d, f, e, k = cfg.n_tok, cfg.d_model, cfg.d_ff, cfg.n_exp, cfg.top_k
        r, fs = cfg.rows, cfg.d_ff_shared
        z = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        # gather=True (inference, bf16 experts, no capacity): GEMM1 reads its rows
        # straight from x (moe_permute_maps + moe_grouped_ffn_gather), no x_perm
        self.gather = gather and (not train) and cfg.precision == "bf16" and cfg.capacity_factor <= 0
        self.checkpoint = checkpoint
        mine = share is None          # buffers in passing are this layer's own
        keep = train and not checkpoint
        self.buf = {
            "logits": z(n, e, dt=F32), "topk_idx": z(n, k, dt=I32), "topk_w": z(n, k, dt=F32),
            "counts": z(e, dt=I32), "offsets": z(e + 1, dt=I32), "row_of_copy": z(r, dt=I32),
            "copy_of_row": z(r, dt=I32), "x_perm": None if self.gather or not mine else z(r, d),
            "h": None if checkpoint else z(r, f), "y_perm": z(r, d) if mine else None, "out": z(n, d),
            "a1": z(r, f) if keep else None, "a3": z(r, f) if keep else None,
        }
        if cfg.n_shared:
            self.buf.update(hs=None if checkpoint else z(n, fs), y_shared=z(n, d) if mine else None,
                            a1s=z(n, fs) if keep else None, a3s=z(n, fs) if keep else None)
        else:
            self.buf.update(hs=None, y_shared=None, a1s=None, a3s=None)
        self.w8 = cfg.precision == "fp8w"
        self.f8 = cfg.precision == "fp8b"
        self.w8q = quantize_weights_fp8_tile(params) if self.w8 or self.f8 else None
        self.cap = cfg.capacity_factor > 0
        if self.cap:
            if cfg.precision in ("mxfp8", "fp8b"):
                raise ValueError("the capacity-factor mode runs with bf16 operands")
            # routing writes the dropless offsets here; b["offsets"] holds the kept ones
            self.buf.update(offsets_full=z(e + 1, dt=I32), row_of_copy_full=z(r, dt=I32),
                            copy_of_row_full=z(r, dt=I32), n_dropped=z(1, dt=I32))
        self.mx = cfg.precision == "mxfp8"
        # E <= 32, bf16 rows, dropless, permuted copy: routing and dispatch in
        # one launch (moe_route_permute); fused_dispatch=False keeps two calls
        self.fused_dispatch = (fused_dispatch and e <= 32 and not self.mx and not self.f8 and not self.cap
                               and not self.gather)
        if self.f8:
            if not train:   # the weight gradients alone read the bf16 rows
                self.buf.update(x_perm=None, h=None, hs=None)
            ld = fp8_scale_ld(d)
            sh = cfg.n_shared
            self.buf.update(xq_perm=z(r, d, dt=U8), xs_perm=z(r, ld, dt=F32), xq_tok=z(n, d, dt=U8) if sh else None,
                            xs_tok=z(n, ld, dt=F32) if sh else None)
        if self.mx:
            self.wq = quantize_weights_mxfp8(params)
            self.wqt = quantize_weights_mxfp8_t(params) if train else None
            self.buf.update(xq_perm=z(r, d, dt=U8), xs_perm=torch.zeros(d // 32, mx_scale_ld(r), dtype=U8, device=device),
                            xq_tok=z(n, d, dt=U8) if cfg.n_shared else None,
                            xs_tok=(torch.zeros(d // 32, mx_scale_ld(n), dtype=U8, device=device)
                                    if cfg.n_shared else None))
        self.ckpt = ckpt_buffers(self.desc, device) if checkpoint else None
        if share is not None:
            self.buf.update({key: share.buf[key] for key in ("x_perm", "y_perm", "y_shared")})
            self.ws = share.ws
        else:
            fwd_b, bwd_b = moe_workspace_size(self.desc)
            need = moe_ckpt_workspace_size(self.desc) if checkpoint else bwd_b if train else fwd_b
            self.ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
            moe_workspace_init(self.ws)
        self.balance = None
        self.grads = None
        if train:
            self.grads = {"dx": z(n, d), "dw_gate": z(e, d, dt=F32), "dw1": z(e, f, d, dt=F32),
                          "dw3": z(e, f, d, dt=F32), "dw2": z(e, d, f, dt=F32), "dg": z(n, k, dt=F32),
                          "dlogits": z(n, k, dt=F32)}
            if cfg.n_shared:
                self.grads.update(dws1=z(fs, d, dt=F32), dws3=z(fs, d, dt=F32), dws2=z(d, fs, dt=F32))
        self.x = None
        self.kept = False   # checkpoint: what a forward kept is there

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        self.experts(x, stream)
        return self._combine(stream)

    def _combine(self, stream=None):
        b = self.buf
        moe_combine(self.desc, b["y_perm"], b["row_of_copy"], b["topk_w"], b["y_shared"], b["out"], stream)
        return b["out"]

    def experts(self, x: torch.Tensor, stream=None):
        """Everything of the forward but the combine: ``buf`` then holds y_perm,
        row_of_copy, topk_w and y_shared."""
        b, p = self.buf, self.p
        self.x = None if self.checkpoint else x
        if self.balance is not None:
            self.balance.pop("pending", None)   # a loss of the forward before, never taken back
        if self.fused_dispatch:
            # routing and the permuted copy of the tokens in one launch (E <= 32)
            moe_route_permute(self.desc, x, p["w_gate"], p.get("bias"), b["logits"], b["topk_idx"], b["topk_w"],
                              b["counts"], b["offsets"], b["row_of_copy"], b["copy_of_row"], b["x_perm"], self.ws,
                              stream)
            return self._ffn(x, stream)
        moe_route(self.desc, x, p["w_gate"], p.get("bias"), b["logits"], b["topk_idx"], b["topk_w"], b["counts"],
                  b["offsets_full"] if self.cap else b["offsets"], self.ws, stream)
        if self.mx:
            return self._experts_mx(x, stream)
        if self.f8:
            return self._experts_fp8b(x, stream)
        if self.gather:
            b = self.buf
            moe_permute_maps(self.desc, b["topk_idx"], b["offsets"], b["row_of_copy"], b["copy_of_row"], self.ws,
                             stream)
            moe_grouped_ffn_gather(self.desc, x, b["copy_of_row"], b["offsets"], p["w1"], p["w3"], p["w2"],
                                   p.get("ws1"), p.get("ws3"), p.get("ws2"), None, None, b["h"], None, None,
                                   b["hs"], b["y_perm"], b["y_shared"], self.ws, stream)
            return
        self._permute(x, stream)
        self._ffn(x, stream)

    def _permute(self, x, stream=None):
        b = self.buf
        if self.cap:
            moe_permute_capacity(self.desc, x, b["topk_idx"], b["offsets_full"], self.cfg.capacity_factor,
                                 b["row_of_copy_full"], b["copy_of_row_full"], b["offsets"], b["row_of_copy"],
                                 b["copy_of_row"], b["x_perm"], b["n_dropped"], self.ws, stream)
        else:
            moe_permute(self.desc, x, b["topk_idx"], b["offsets"], b["row_of_copy"], b["copy_of_row"], b["x_perm"],
                        self.ws, stream)

    def _ffn(self, x, stream=None):
        b, p = self.buf, self.p
        if self.checkpoint:
            moe_quantize_mxfp8(x, self.ckpt["x"], self.ckpt["x_scale"], stream)
            moe_grouped_ffn_ckpt(self.desc, b["x_perm"], b["offsets"], x, p, self.ckpt, b["y_perm"], b["y_shared"],
                                 self.ws, stream)
            self.kept = True
        elif self.w8:
            saved = {key: b[key] for key in ("a1", "a3", "h", "a1s", "a3s", "hs") if b.get(key) is not None}
            moe_grouped_ffn_fp8w(self.desc, b["x_perm"], b["offsets"], x, self.w8q, saved, b["y_perm"],
                                 b["y_shared"], self.ws, stream)
        else:
            moe_grouped_ffn(self.desc, b["x_perm"], b["offsets"], x, p["w1"], p["w3"], p["w2"], p.get("ws1"),
                            p.get("ws3"), p.get("ws2"), b["a1"], b["a3"], b["h"], b["a1s"], b["a3s"], b["hs"],
                            b["y_perm"], b["y_shared"], self.ws, stream)

    def _ffn_combine(self, x, stream=None):
        self._ffn(x, stream)
        return self._combine(stream)

    def _forward_mx(self, x, stream=None):
        self._experts_mx(x, stream)
        return self._combine(stream)

    def _experts_mx(self, x, stream=None):
        b = self.buf
        moe_permute_mxfp8(self.desc, x, b["topk_idx"], b["offsets"], b["row_of_copy"], b["copy_of_row"],
                          b["xq_perm"], b["xs_perm"], b["xq_tok"], b["xs_tok"], self.ws, stream)
        saved = ({key: b[key] for key in ("a1", "a3", "h", "a1s", "a3s", "hs") if b.get(key) is not None}
                 if self.train else {})
        moe_grouped_ffn_mxfp8(self.desc, b["xq_perm"], b["xs_perm"], b["offsets"], b["xq_tok"], b["xs_tok"], self.wq,
                              saved, b["y_perm"], b["y_shared"], self.ws, stream)

    def _experts_fp8b(self, x, stream=None):
        b = self.buf
        moe_permute_fp8b(self.desc, x, b["topk_idx"], b["offsets"], b["row_of_copy"], b["copy_of_row"], b["x_perm"],
                         b["xq_perm"], b["xs_perm"], b["xq_tok"], b["xs_tok"], self.ws, stream)
        saved = ({key: b[key] for key in ("a1", "a3", "h", "a1s", "a3s", "hs") if b.get(key) is not None}
                 if self.train else {})
        moe_grouped_ffn_fp8b(self.desc, b["xq_perm"], b["xs_perm"], b["offsets"], b["xq_tok"], b["xs_tok"], self.w8q,
                             saved, b["y_perm"], b["y_shared"], self.ws, stream)

    def balance_loss(self, seq_offsets: torch.Tensor, coef: float, z_coef: float = 0.0, dloss=None,
                     stream=None) -> torch.Tensor:
        """The balance and z losses (fp32 [2]) of the last forward's routing over the sequences
        ``seq_offsets`` (int32 [S + 1]); the next backward adds their gradient, times ``dloss``, to dx and
        dw_gate.  ``balance["counts"]`` holds the copies per sequence and expert."""
        if not self.train:
            raise ValueError("a layer built with train=False has no backward")
        if self.cap:
            raise ValueError("the balance over sequences is of the dropless layer")
        self._needs_forward("balance_loss")
        b, e = self.buf, self.cfg.n_exp
        s = seq_offsets.shape[0] - 1
        z = lambda *shape, dt: torch.empty(shape, dtype=dt, device=b["logits"].device)  # noqa: E731
        if self.balance is None:
            self.balance = {"loss": z(2, dt=F32), "dlogits": z(self.cfg.n_tok, e, dt=F32)}
            self._counts = []
        # room for twice as many sequences whenever it grows; captured steps go on writing where they did
        if not self._counts or self._counts[-1].shape[0] < s:
            self._counts.append(z(max(s, 2 * self._counts[-1].shape[0]) if self._counts else s, e, dt=I32))
        self.balance["counts"] = self._counts[-1][:s]
        q = self.balance
        moe_balance_loss(self.desc, b["logits"], b["topk_idx"], seq_offsets, q["counts"], q["loss"], q["dlogits"],
                         self.ws, coef, z_coef, dloss, stream)
        q["pending"] = True
        return q["loss"]

    def _needs_forward(self, what: str):
        # buffers that no forward has written hold any index
        if self.x is None and not self.kept:
            raise ValueError(f"{what} needs the forward that it belongs to")

    def backward(self, dy: torch.Tensor, stream=None) -> dict:
        if not self.train:
            raise ValueError("a layer built with train=False has no backward")
        self._needs_forward("backward")
        self._backward(dy, stream)
        q, g = self.balance, self.grads
        if q is not None and q.pop("pending", False):
            x = self.x
            if self.checkpoint:   # decoded where the forward's permuted rows were
                x = self.buf["x_perm"][:self.cfg.n_tok]
                moe_dequantize_mxfp8(self.ckpt["x"], self.ckpt["x_scale"], x, stream)
            moe_router_backward(self.desc, q["dlogits"], x, self.p["w_gate"], g["dx"], g["dx"], g["dw_gate"],
                                g["dw_gate"], self.ws, stream)
        return g

    def _backward(self, dy: torch.Tensor, stream=None) -> dict:
        b = self.buf
        if self.checkpoint:
            state = {key: b[key] for key in ("logits", "topk_idx", "topk_w", "offsets", "row_of_copy",
                                             "copy_of_row")}
            moe_backward_ckpt(self.desc, self.p["w_gate"], self.p, {**state, **self.ckpt}, dy, self.grads, self.ws,
                              stream)
            return self.grads
        if self.mx:
            state = {key: b[key] for key in ("logits", "topk_idx", "topk_w", "offsets", "row_of_copy",
                                             "copy_of_row", "a1", "a3", "h", "y_perm", "a1s", "a3s", "hs")}
            state["x"] = self.x
            moe_backward_mxfp8(self.desc, self.p["w_gate"], self.wqt, state, dy, self.grads, self.ws, stream)
            return self.grads
        state = {key: b[key] for key in ("x_perm", "logits", "topk_idx", "topk_w", "offsets", "row_of_copy",
                                         "copy_of_row", "a1", "a3", "h", "y_perm", "a1s", "a3s", "hs")}
        state["x"] = self.x
        if self.cap:
            state.update(offsets_full=b["offsets_full"], copy_of_row_full=b["copy_of_row_full"])
        if self.f8:
            moe_backward_fp8b(self.desc, self.p["w_gate"], self.w8q, state, dy, self.grads, self.ws, stream)
        elif self.w8:
            moe_backward_fp8w(self.desc, self.p["w_gate"], self.w8q, state, dy, self.grads, self.ws, stream)
        else:
            moe_backward(self.desc, self.p["w_gate"], self.p, state, dy, self.grads, self.ws, stream)
        return self.grads

    def drop_rate(self) -> float:
        """Fraction of token copies dropped by the capacity in the last forward (0 when dropless)."""
        if not self.cap:
            return 0.0
        return int(self.buf["n_dropped"].item()) / self.cfg.rows

    def update_bias(self, gamma: float = 1e-3, mode: int = 0, stream=None):
        moe_update_bias(self.desc, self.buf["counts"], self.p["bias"], gamma, mode, stream)

    def device_status(self) -> tuple[int, int]:
        return moe_get_device_status(self.ws)


class MoEBlock:
    """A pre-norm block around one layer: out = x + dropout(MoE(layernorm(x))).

    ``gamma``, ``beta``: fp32 [D] (beta may be None).  The residual stream x is
    bf16 or fp32 (``stream_dtype``).  ``rng`` (seed, offset) lives on the
    device; every training forward that drops moves the offset past the counters it used, as an
    ordinary tensor operation on the same stream, so a captured step draws anew
    at each replay.  ``backward`` uses the offset of the last forward.
    ``checkpoint``: the layer keeps its activations in 8 bits (:class:`MoELayer`).
    """

    def __init__(self, cfg: MoEConfig, params: dict, gamma, beta=None, p: float = 0.0, seed: int = 0,
                 eps: float = 1e-5, train: bool = True, stream_dtype=BF16, device="cuda", checkpoint: bool = False):
        if not 0.0 <= p < 1.0:
            raise ValueError(f"p must be in [0, 1), got {p}")
        self.layer = MoELayer(cfg, params, train=train, device=device, checkpoint=checkpoint)
        self.desc, self.train, self.p, self.eps = self.layer.desc, train, float(p), float(eps)
        self.gamma, self.beta = gamma, beta
        n, d = cfg.n_tok, cfg.d_model
        z = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.normed, self.out = z(n, d), z(n, d, dt=stream_dtype)
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=device)
        self.used = torch.zeros(2, dtype=torch.int64, device=device)
        self.step = torch.tensor([0, (n * d + 3) // 4], dtype=torch.int64, device=device)
        self.mean = self.rstd = self.grads = None
        if train:
            self.mean, self.rstd, self.dmoe = z(n, dt=F32), z(n, dt=F32), z(n, d)
            self.grads = {"dx": z(n, d, dt=stream_dtype), "dgamma": z(d, dt=F32),
                          "dbeta": z(d, dt=F32) if beta is not None else None}
        self.x = None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        b = self.layer.buf
        p = self.p if self.train else 0.0
        self.x = x
        moe_layernorm(self.desc, x, self.gamma, self.beta, self.normed, self.mean, self.rstd, self.eps)
        self.layer.experts(self.normed)
        if p > 0.0:
            self.used.copy_(self.rng)
            self.rng.add_(self.step)
        moe_combine_dropout(self.desc, b["y_perm"], b["row_of_copy"], b["topk_w"], b["y_shared"], x, self.used, p,
                            self.out)
        return self.out

    def backward(self, dout: torch.Tensor) -> dict:
        """``dout`` of the residual stream's type; returns dx, dgamma, dbeta and,
        under "layer", the gradients of :meth:`MoELayer.backward`.  Needs ``train`` and a forward."""
        if not self.train:
            raise ValueError("a block built with train=False has no backward")
        if self.x is None:
            raise ValueError("backward needs the forward that it belongs to")
        g = self.grads
        moe_dropout_backward(self.desc, dout, self.used, self.p, self.dmoe)
        inner = self.layer.backward(self.dmoe)
        moe_layernorm_backward(self.desc, inner["dx"], self.x, self.gamma, self.mean, self.rstd, dout, g["dx"],
                               g["dgamma"], g["dbeta"], self.layer.ws)
        return {**g, "layer": inner}

    def device_status(self) -> tuple[int, int]:
        return self.layer.device_status()
