"""Refusals of the block's entry points, on the CPU: every error the host can
detect returns before anything is enqueued (the addresses are never read)."""
import ctypes

import pytest
import torch

from ragged_grouped_gemm_gb300 import _lib, api, build
from ragged_grouped_gemm_gb300.inputs import CONFIGS

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20          # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _desc(**kw):
    d = api.make_desc(CONFIGS["tiny"])
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _ws(lib, d):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_workspace_size(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)) == OK
    return f.value, b.value


def test_workspace_of_the_fp8_layer(lib):
    plain, fp8 = _ws(lib, _desc()), _ws(lib, _desc(precision=4))
    assert fp8[0] > plain[0] and fp8[1] > plain[1]
    assert api.make_desc(CONFIGS["tiny"].replace(precision="fp8b")).precision == 4


@pytest.mark.parametrize("rows,cols,ld,src,codes,scales,want", [
    (4, 100, 4, P, P, P, INVALID), (4, 0, 4, P, P, P, INVALID), (4, 256, 1, P, P, P, INVALID),
    (-1, 256, 4, P, P, P, INVALID), (4, 256, 4, None, P, P, INVALID), (4, 256, 4, P + 8, P, P, INVALID),
    (4, 256, 4, P, P + 4, P, INVALID), (4, 256, 4, P, P, None, INVALID), (4, 256, 4, P, P, P + 2, INVALID),
    (0, 256, 4, None, None, None, OK)])
def test_quantize_rows_refusals(lib, rows, cols, ld, src, codes, scales, want):
    assert lib.moe_quantize_fp8_rows(src, rows, cols, codes, scales, ld, None) == want


def test_grouped_gemm_refusals(lib):
    def call(g=4, rows=8, n=64, k=128, a=P, sa=P, ld=4, off=P, b=P, sb=P, mn=0, out=P, ws=P, wsb=1 << 20):
        return lib.moe_grouped_gemm_fp8(g, rows, n, k, a, sa, ld, off, b, sb, mn, out, ws, wsb, None)
    for bad in (dict(g=0), dict(g=1025), dict(rows=-1), dict(n=0), dict(k=0), dict(n=72), dict(k=72),
                dict(ld=0), dict(k=144, ld=1), dict(ld=5), dict(sa=P + 8), dict(mn=2), dict(a=None), dict(a=P + 8), dict(b=P + 4),
                dict(out=P + 2), dict(sa=None), dict(sb=None), dict(off=None), dict(rows=1 << 31),
                dict(n=1 << 30), dict(k=1 << 30)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=P + 8), dict(wsb=16)):
        assert call(**bad) == WORKSPACE, bad
    assert call(rows=0) == OK
    b = ctypes.c_size_t()
    assert lib.moe_grouped_gemm_fp8_workspace_size(4, 8, 64, 128, None) == INVALID
    assert lib.moe_grouped_gemm_fp8_workspace_size(4, 8, 64, 128, ctypes.byref(b)) == OK and b.value >= 256


def test_layer_entry_refusals(lib):
    d = _desc(precision=4)
    f, b = _ws(lib, d)
    ref = ctypes.byref(d)
    w = _lib.MoeExpertWeightsMx(*[P] * 12)
    sv = _lib.MoeFfnSaved(*[P] * 6)
    ffn = lambda desc=ref, xq=P, ww=w, s=sv, ws=P, n=f: lib.moe_grouped_ffn_fp8b(  # noqa: E731
        desc, xq, P, P, None, None, ctypes.byref(ww), ctypes.byref(s), P, None, ws, n, None)
    assert ffn(xq=None) == INVALID and ffn(xq=P + 8) == INVALID
    assert ffn(ws=None) == WORKSPACE and ffn(n=f - 1) == WORKSPACE
    assert ffn(desc=ctypes.byref(_desc())) == INVALID                     # another precision
    assert ffn(ww=_lib.MoeExpertWeightsMx(*([P, None] + [P] * 10))) == INVALID
    assert ffn(s=_lib.MoeFfnSaved(P + 8, P, P, P, P, P)) == INVALID
    perm = lambda desc=ref, x=P, xt=None, st=None, ws=P: lib.moe_permute_fp8b(  # noqa: E731
        desc, x, P, P, P, P, None, P, P, xt, st, ws, f, None)
    assert perm(x=None) == INVALID and perm(xt=P, st=None) == INVALID and perm(ws=None) == WORKSPACE
    assert perm(desc=ctypes.byref(_desc(precision=2))) == INVALID
    st, g = _lib.MoeFwdState(*[P] * 17), _lib.MoeGrads(*[P] * 10)
    bwd = lambda desc=ref, ww=ctypes.byref(w), n=b: lib.moe_backward_fp8b(  # noqa: E731
        desc, P, ww, ctypes.byref(st), P, ctypes.byref(g), P, n, None)
    assert bwd(desc=ctypes.byref(_desc())) == INVALID and bwd(ww=None) == INVALID and bwd(n=f) == WORKSPACE
    # the other entry points do not take the FP8 layer
    plain = _lib.MoeExpertWeights(*[P] * 6)
    assert lib.moe_grouped_ffn(ref, P, P, P, ctypes.byref(plain), ctypes.byref(sv), P, P, P, f, None) == UNSUPPORTED
    assert lib.moe_backward(ref, P, ctypes.byref(plain), ctypes.byref(st), P, ctypes.byref(g), P, b, None) == UNSUPPORTED


def test_layernorm_refusals(lib):
    d = _desc()
    _, b = _ws(lib, d)

    def fwd(desc=d, x=P, f32=0, gamma=P, beta=None, eps=1e-5, y=P):
        return lib.moe_layernorm(ctypes.byref(desc), x, f32, gamma, beta, eps, y, None, None, None)
    for bad in (dict(x=None), dict(x=P + 8), dict(f32=2), dict(gamma=None), dict(beta=P + 4), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-60), dict(y=None)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(desc=_desc(d_model=32768 + 64)) == UNSUPPORTED
    assert fwd(desc=_desc(n_tok=0), x=None, y=None) == OK

    def bwd(dy=P, f32=0, mean=P, rstd=P, dres=None, dgamma=P, ws=P, n=b):
        return lib.moe_layernorm_backward(ctypes.byref(d), dy, P, f32, P, mean, rstd, dres, P, dgamma, P, ws, n, None)
    for bad in (dict(dy=None), dict(f32=3), dict(mean=None), dict(rstd=None), dict(dres=P + 8), dict(dgamma=None)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(ws=None) == WORKSPACE and bwd(n=b - 1) == WORKSPACE


def test_dropout_refusals(lib):
    d = _desc()

    def fwd(desc=d, y=P, p=0.1, f32=0, resid=P, rng=P, out=P, ys=None):
        return lib.moe_combine_dropout(ctypes.byref(desc), y, P, P, ys, resid, f32, rng, p, out, None)
    for bad in (dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(f32=2), dict(rng=None), dict(rng=P + 4),
                dict(out=None), dict(y=P + 8), dict(resid=P + 8), dict(ys=P + 8)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(desc=_desc(n_tok=0), y=None, out=None) == OK

    def bwd(dout=P, p=0.1, f32=0, rng=P, dy=P):
        return lib.moe_dropout_backward(ctypes.byref(d), dout, f32, rng, p, dy, None)
    for bad in (dict(dout=None), dict(p=1.5), dict(f32=-1), dict(rng=None), dict(dy=P + 4)):
        assert bwd(**bad) == INVALID, bad


def test_binding_refuses_wrong_tensors():
    d = _desc()
    x = torch.zeros(d.n_tok, d.d_model, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.moe_layernorm(d, x, x, None, x)
    with pytest.raises(ValueError, match="three dimensions"):
        api.moe_grouped_gemm_fp8(x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="p must be"):
        api.MoEBlock(CONFIGS["tiny"], {}, None, p=1.0, device="cpu")
