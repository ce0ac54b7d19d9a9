"""Refusals of the balance loss, the dense router gradient and the 8-bit checkpoints.  Every call is refused before
anything is enqueued (the addresses are never read)."""
import ctypes
import subprocess

import pytest
import torch

from ragged_grouped_gemm_gb300 import _lib, api, build
from ragged_grouped_gemm_gb300.inputs import CONFIGS, MoEConfig

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 1 << 20          # an aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _desc(name="tiny", **kw):
    d = api.make_desc(CONFIGS[name])
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _ws(lib, d):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_workspace_size(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)) == 0
    return f.value, b.value


def test_structs_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe.h"', "int main(void) {"]
    want = []
    for cname, py in (("moe_ckpt_t", _lib.MoeCkpt), ("moe_ckpt_state_t", _lib.MoeCkptState)):
        lines.append(f'  printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for name, _ in py._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({cname}, {name}));')
            want.append(getattr(py, name).offset)
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["  return 0; }"]))
    subprocess.run(["gcc", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    assert [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want


def test_balance_loss_refusals(lib):
    def call(d=_desc(), logits=P, idx=P, off=P, n=3, coef=0.1, z=0.1, dloss=None, counts=P, loss=P, dl=P, ws=P,
             nb=BIG):
        return lib.moe_balance_loss(ctypes.byref(d), logits, idx, off, n, coef, z, dloss, counts, loss, dl, ws, nb, None)
    for bad in (dict(logits=None), dict(idx=None), dict(off=None), dict(counts=None), dict(loss=None), dict(n=0),
                dict(n=-1), dict(n=(1 << 24) + 1), dict(coef=float("nan")), dict(z=float("inf")), dict(logits=P + 2),
                dict(idx=P + 1), dict(off=P + 2), dict(dloss=P + 2), dict(counts=P + 3), dict(loss=P + 2),
                dict(dl=P + 2), dict(d=_desc(top_k=9)), dict(d=_desc(gate=2))):
        assert call(**bad) == INVALID, bad
    assert call(nb=_ws(lib, _desc())[0] - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(ws=P + 8) == WORKSPACE


def test_router_backward_refusals(lib):
    def call(d=_desc(), dl=P, x=P, wg=P, dxi=None, dx=P, dwi=None, dw=P, ws=P, nb=BIG):
        return lib.moe_router_backward(ctypes.byref(d), dl, x, wg, dxi, dx, dwi, dw, ws, nb, None)
    for bad in (dict(dl=None), dict(x=None), dict(wg=None), dict(dx=None), dict(dw=None), dict(dl=P + 4),
                dict(x=P + 2), dict(wg=P + 8), dict(dxi=P + 8), dict(dx=P + 2), dict(dwi=P + 4), dict(dw=P + 4)):
        assert call(**bad) == INVALID, bad
    assert call(nb=_ws(lib, _desc())[1] - 1) == WORKSPACE and call(ws=None) == WORKSPACE


@pytest.mark.parametrize("n,d,e", [(1, 64, 1), (1, 64, 1024), (7, 7168, 1000), (4096, 64, 256), (300, 4096, 1021)])
def test_router_scratch_fits_the_workspace(lib, n, d, e):
    """Terms of dlogits and one run's partial gradient, over the layer's own scratch or behind it."""
    c = MoEConfig("case", n, d, 64, e, 1)
    e8 = (e + 7) // 8 * 8
    need = n * 3 * e8 * 2 + 256 + (3 * e8 if 3 * e8 <= 128 else e8) * d * 4
    assert _ws(lib, api.make_desc(c))[1] >= need


def test_checkpoint_layer_refusals(lib):
    d = _desc(n_shared=1, d_ff_shared=64)
    size = ctypes.c_size_t()
    assert lib.moe_ckpt_workspace_size(ctypes.byref(d), ctypes.byref(size)) == 0
    assert size.value > _ws(lib, d)[1]
    assert lib.moe_ckpt_workspace_size(ctypes.byref(d), None) == INVALID
    for precision in (1, 2, 4):
        q = _desc(precision=precision)
        assert lib.moe_ckpt_workspace_size(ctypes.byref(q), ctypes.byref(size)) == UNSUPPORTED
    w = [P] * 6
    kept = [P] * 8

    def fwd(desc=d, x_perm=P, off=P, x=P, w=w, kept=kept, y=P, ys=P, ws=P, nb=BIG):
        return lib.moe_grouped_ffn_ckpt(ctypes.byref(desc), x_perm, off, x, ctypes.byref(_lib.MoeExpertWeights(*w)),
                                        ctypes.byref(_lib.MoeCkpt(*kept)), y, ys, ws, nb, None)

    def bwd(desc=d, wg=P, w=w, st=[P] * 8, kept=kept, dy=P, grads=[P] * 10, ws=P, nb=BIG):
        state = _lib.MoeCkptState(*st, _lib.MoeCkpt(*kept))
        return lib.moe_backward_ckpt(ctypes.byref(desc), wg, ctypes.byref(_lib.MoeExpertWeights(*w)),
                                     ctypes.byref(state), dy, ctypes.byref(_lib.MoeGrads(*grads)), ws, nb, None)
    for bad in (dict(x_perm=None), dict(off=None), dict(off=P + 2), dict(x=None), dict(y=None), dict(ys=None),
                dict(y=P + 8)):
        assert fwd(**bad) == INVALID, bad
    for i in range(8):
        for v in (None, P + 8):
            some = [v if j == i else P for j in range(8)]
            assert fwd(kept=some) == INVALID and bwd(kept=some) == INVALID, i
            word = v if i < 2 or v is None else P + 2       # x and its scales, then arrays of 32-bit numbers
            assert bwd(st=[word if j == i else P for j in range(8)]) == INVALID, i
    for i in range(6):
        some = [None if j == i else P for j in range(6)]
        assert fwd(w=some) == INVALID and bwd(w=some) == INVALID, i
    for i in range(8):                         # dg and dlogits (8, 9) may be null
        assert bwd(grads=[None if j == i else P for j in range(10)]) == INVALID, i
    for i in (8, 9):
        assert bwd(grads=[P + 2 if j == i else P for j in range(10)]) == INVALID, i
    assert bwd(wg=None) == INVALID and bwd(dy=P + 2) == INVALID
    need = ctypes.c_size_t()
    lib.moe_ckpt_workspace_size(ctypes.byref(d), ctypes.byref(need))
    for call in (fwd, bwd):
        assert call(nb=need.value - 1) == WORKSPACE and call(ws=None) == WORKSPACE
        assert call(desc=_desc(precision=4)) == UNSUPPORTED


def test_kept_products_refusals(lib):
    size = ctypes.c_size_t()

    def swiglu(g=4, rows=100, d=128, f=64, dy=P, off=P, w2=P, rw=None, a1=P, a1s=P, a3=P, a3s=P, ld=112, o=(P, P, P),
               dg=None, ws=P, nb=BIG):
        return lib.moe_swiglu_backward_ckpt(g, rows, d, f, dy, off, w2, rw, a1, a1s, a3, a3s, ld, *o, dg, ws, nb, None)
    for bad in (dict(g=0), dict(g=1025), dict(rows=-1), dict(d=100), dict(f=32), dict(d=0), dict(rows=1 << 31), dict(ld=99),
                dict(ld=104), dict(dy=None), dict(off=None), dict(off=P + 1), dict(w2=P + 8), dict(rw=P + 2),
                dict(a1=None), dict(a1s=P + 4), dict(a3=P + 1), dict(a3s=None), dict(o=(None, P, P)),
                dict(o=(P, P + 8, P)), dict(o=(P, P, None)), dict(dg=P + 2)):
        assert swiglu(**bad) == INVALID, bad
    assert lib.moe_swiglu_backward_ckpt_workspace_size(4, 100, 128, 64, ctypes.byref(size)) == 0
    assert swiglu(nb=size.value - 1) == WORKSPACE and swiglu(ws=P + 8) == WORKSPACE
    assert swiglu(rows=0, ld=0, dy=None) == 0        # nothing to do

    def wgrad(g=4, rows=100, m=128, k=64, dy=P, x=P, xs=P, n=50, ld=64, rm=P, div=2, off=P, dw=P, ws=P, nb=BIG):
        return lib.moe_grouped_wgrad_ckpt(g, rows, m, k, dy, x, xs, n, ld, rm, div, off, dw, ws, nb, None)
    for bad in (dict(g=0), dict(g=1025), dict(rows=-1), dict(m=100), dict(k=96), dict(ld=48), dict(ld=52), dict(n=-1),
                dict(div=0), dict(rm=None), dict(rm=None, n=100, ld=112), dict(rm=None, div=1), dict(rm=P + 2),
                dict(dy=None), dict(x=None), dict(xs=P + 8), dict(off=P + 2), dict(dw=None), dict(dw=P + 4)):
        assert wgrad(**bad) == INVALID, bad
    assert lib.moe_grouped_wgrad_ckpt_workspace_size(4, 100, 128, 64, ctypes.byref(size)) == 0
    assert wgrad(nb=size.value - 1) == WORKSPACE and wgrad(ws=None) == WORKSPACE

    def deq(c=P, s=P, rows=5, cols=64, ld=16, o=P):
        return lib.moe_dequantize_mxfp8(c, s, rows, cols, ld, o, None)
    for bad in (dict(c=None), dict(s=P + 8), dict(o=None), dict(rows=-1), dict(cols=0), dict(cols=48), dict(ld=0), dict(ld=8)):
        assert deq(**bad) == INVALID, bad
    assert deq(rows=0, c=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    d = _desc()
    with pytest.raises(ValueError, match="CUDA"):
        api.moe_balance_loss(d, torch.zeros(256, 8), None, torch.zeros(3, dtype=torch.int32), None, None)
    with pytest.raises(ValueError, match="seq_offsets"):
        api.moe_balance_loss(d, None, None, torch.zeros(1, dtype=torch.int32), None, None)
    with pytest.raises(ValueError, match="three dimensions"):
        api.moe_swiglu_backward_ckpt(None, None, torch.zeros(2, 2), None, None, torch.zeros(2, 2), *[None] * 7)
    with pytest.raises(ValueError, match="three dimensions"):
        api.moe_grouped_wgrad_ckpt(None, None, torch.zeros(2, 2), None, None, 1, torch.zeros(2, 2), None)


@pytest.mark.parametrize("kw", [dict(train=False), dict(precision="mxfp8"), dict(precision="fp8w"),
                                dict(precision="fp8b"), dict(capacity_factor=1.0)])
def test_layer_refuses_checkpoints_it_has_not(kw):
    train = kw.pop("train", True)
    with pytest.raises(ValueError, match="checkpoints"):
        api.MoELayer(CONFIGS["tiny"].replace(**kw), {}, train=train, checkpoint=True, device="cpu")
