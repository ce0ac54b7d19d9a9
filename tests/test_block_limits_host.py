"""Limits of the block's entry points and kernels that hold on the CPU.  Every call
here is refused before anything is enqueued (the addresses are never read)."""
import ctypes
import glob
import os
import re

import pytest

from ragged_grouped_gemm_gb300 import _lib, api, build
from ragged_grouped_gemm_gb300.inputs import CONFIGS

INVALID = 1
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
    assert lib.moe_workspace_size(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)) == 0
    return f.value, b.value


def _sources():
    return {os.path.basename(p): open(p).read() for p in glob.glob(os.path.join(build.CSRC, "*.cu*"))}


def test_every_aligned_cluster_barrier_converges_its_warp_first():
    """`barrier.cluster.*.aligned` is undefined for a warp whose lanes do not arrive together, and a
    branch of some lanes may stand right before any call: the convergence belongs to the barrier's
    own wrapper, and no other code issues it."""
    found = []
    for name, text in _sources().items():
        for m in re.finditer(r"barrier\.cluster\.arrive", text):
            body = text[text.rfind("{", 0, m.start()):m.start()]
            found.append(name)
            assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"$", body), (name, body)
    assert found == ["sm100_ptx.cuh"]


@pytest.mark.parametrize("odd", [1, 2, 3])
def test_misaligned_arrays_of_32_bit_numbers_are_refused(lib, odd):
    """The kernels read them word by word: an address between two words would fault on the device."""
    q = P + odd
    for off, sb in ((q, P), (P, q)):
        assert lib.moe_grouped_gemm_fp8(4, 8, 64, 128, P, P, 4, off, P, sb, 0, P, P, 1 << 20, None) == INVALID
    d = _desc(precision=4, n_shared=1, d_ff_shared=64)
    f, b = _ws(lib, d)
    ref = ctypes.byref(d)
    for i in range(4):
        maps = [q if i == j else P for j in range(4)]
        assert lib.moe_permute_fp8b(ref, P, maps[0], maps[1], maps[2], maps[3], None, P, P, None, None, P, f,
                                    None) == INVALID
    saved = ctypes.byref(_lib.MoeFfnSaved(*[P] * 6))
    state, grads = ctypes.byref(_lib.MoeFwdState(*[P] * 17)), ctypes.byref(_lib.MoeGrads(*[P] * 10))
    plain = ctypes.byref(_lib.MoeExpertWeightsMx(*[P] * 12))
    assert lib.moe_grouped_ffn_fp8b(ref, P, P, q, P, P, plain, saved, P, P, P, f, None) == INVALID
    for i in range(6):
        w = ctypes.byref(_lib.MoeExpertWeightsMx(*[q if j == 2 * i + 1 else P for j in range(12)]))
        assert lib.moe_grouped_ffn_fp8b(ref, P, P, P, P, P, w, saved, P, P, P, f, None) == INVALID
        assert lib.moe_backward_fp8b(ref, P, w, state, P, grads, P, b, None) == INVALID
    t = _desc()
    ref, b = ctypes.byref(t), _ws(lib, t)[1]
    for mean, rstd in ((q, None), (None, q)):
        assert lib.moe_layernorm(ref, P, 0, P, None, 1e-5, P, mean, rstd, None) == INVALID
    for i in range(4):
        mean, rstd, dgamma, dbeta = (q if i == j else P for j in range(4))
        assert lib.moe_layernorm_backward(ref, P, P, 0, P, mean, rstd, None, P, dgamma, dbeta, P, b, None) == INVALID
    for rows, w in ((q, P), (P, q)):
        assert lib.moe_combine_dropout(ref, P, rows, w, None, None, 0, P, 0.1, P, None) == INVALID


def test_layernorm_timeout_selftest_refusals(lib):
    d = _desc(d_model=2048)
    b = _ws(lib, d)[1]

    def call(desc=d, dy=None, x=P, f32=0, y=P, mean=P, dx=P, dgamma=P, row=0, limit=50_000, ws=P, n=b):
        return lib.moe_selftest_layernorm_timeout(ctypes.byref(desc), dy, x, f32, P, y, mean, P, dx, dgamma, P, row,
                                                  limit, ws, n, None)
    for bad in (dict(x=None), dict(f32=2), dict(y=None), dict(y=P + 8), dict(mean=None), dict(row=-1),
                dict(row=d.n_tok), dict(limit=0), dict(limit=1_000_000_001), dict(dy=P + 8), dict(dy=P, dx=None),
                dict(dy=P, dgamma=None), dict(dy=P, dgamma=P + 2)):
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == 3 and call(n=b - 1) == 3
    for wide in (1024, 32768 + 64):                       # rows that no wait holds up, rows that are too wide
        assert call(desc=_desc(d_model=wide)) == 2


# bytes of the backward workspace of the layer alone
LAYER_BACKWARD_BYTES = [
    ("tiny", "bf16", 1751808),
    ("tiny", "mxfp8", 2597120),
    ("tiny", "fp8w", 1751808),
    ("mixtral", "bf16", 541083136),
    ("mixtral", "mxfp8", 1289373696),
    ("mixtral", "fp8w", 541083136),
    ("dsv3", "bf16", 870979584),
    ("dsv3", "mxfp8", 2575179264),
    ("dsv3", "fp8w", 870979584),
    ("mixtral_quarter", "bf16", 188761600),
    ("mixtral_quarter", "mxfp8", 460179456),
    ("mixtral_quarter", "fp8w", 188761600),
    ("dsv3_e16", "bf16", 49044736),
    ("dsv3_e16", "mxfp8", 155016960),
    ("dsv3_e16", "fp8w", 49044736),
    ("small_softmax", "bf16", 5666304),
    ("small_softmax", "mxfp8", 12626176),
    ("small_softmax", "fp8w", 5666304),
    ("small_sigmoid", "bf16", 9567488),
    ("small_sigmoid", "mxfp8", 22138368),
    ("small_sigmoid", "fp8w", 9567488),
    ("small_fine", "bf16", 8250112),
    ("small_fine", "mxfp8", 29110272),
    ("small_fine", "fp8w", 8250112)]


@pytest.mark.parametrize("name,precision,layer", LAYER_BACKWARD_BYTES)
def test_norm_adds_nothing_to_the_layers_workspace(lib, name, precision, layer):
    """Its partial sums lie over the layer backward's own scratch."""
    assert _ws(lib, api.make_desc(CONFIGS[name].replace(precision=precision)))[1] == layer


def test_norm_workspace_where_the_layers_is_smaller(lib):
    n, d = 16, 32768
    f, b = _ws(lib, _desc(n_tok=n, d_model=d, d_ff=64, n_exp=8, top_k=1))
    assert b - f >= n * 2 * d * 4                     # a partial sum of each gradient for every row


def test_block_backward_without_training_or_forward_is_refused():
    block = api.MoEBlock.__new__(api.MoEBlock)
    block.train, block.x = False, object()
    with pytest.raises(ValueError, match="train=False"):
        block.backward(None)
    block.train, block.x = True, None
    with pytest.raises(ValueError, match="forward"):
        block.backward(None)
