"""Pins of the oracle of the pre-norm block's operators (CPU)."""
import numpy as np
import pytest
import torch

import oracle as O


def test_philox_known_answers():
    # the published test vectors of Philox-4x32-10: counter and key all zero, and all ones in the low halves used here
    assert O.philox_words(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    seen = {tuple(O.philox_words(s, c)) for s in (0, 1, 1 << 33) for c in (0, 1, 1 << 32, (1 << 64) - 1)}
    assert len(seen) == 12                       # seed and both halves of the counter matter


def test_dropout_rate_and_edges():
    n = 40000
    for p in (0.0, 0.1, 0.5):
        kept = O.dropout_keep(5, 77, n, p).mean()
        assert abs(kept - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n)     # five standard deviations
    assert O.dropout_keep(5, 77, 64, 0.0).all()
    # elements of neighbouring calls come from disjoint counters
    a, b = O.dropout_keep(9, 0, 4096, 0.5), O.dropout_keep(9, 1024, 4096, 0.5)
    assert abs((a == b).mean() - 0.5) < 5 * 0.5 / np.sqrt(4096)
    np.testing.assert_array_equal(O.dropout_keep(9, 0, 8192, 0.5)[4096:], b)


def test_fp8_rows_block_edges():
    x = np.zeros((3, 144), np.float32)
    x[0, 0], x[0, 143], x[1, 5] = 448.0, -1.75, 2.0 ** -140
    c, s = O.fp8_rows_quantize(x)
    assert s.shape == (3, 2) and s[0, 0] == 1.0 and s[2, 0] == 1.0 and s[2, 1] == 1.0
    assert c[0, 0] == 0x7E and c[0, 143] == 0xFE and c[2].max() == 0
    v = O.fp8_rows_dequantize(c, s)
    assert v[0, 0] == 448.0 and abs(v[0, 143] + 1.75) <= 2.0 ** -24 * 1.75
    # every value within half a code step: 2^-4 of the value, or half of the smallest code
    x = np.random.default_rng(1).standard_normal((4, 300)).astype(np.float32)
    c, s = O.fp8_rows_quantize(x)
    sf = np.repeat(s, 128, axis=1)[:, :300]
    assert (np.abs(O.fp8_rows_dequantize(c, s) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sf)).all()


@pytest.mark.parametrize("n,d", [(1, 8), (5, 64), (3, 200)])
def test_layernorm_gradient_against_autograd_and_differences(n, d):
    r = np.random.default_rng(n * d)
    x, dy, dres = (r.standard_normal((n, d)) for _ in range(3))
    gamma, beta = r.standard_normal(d), r.standard_normal(d)
    tx, tg, tb = (torch.tensor(v, requires_grad=True) for v in (x, gamma, beta))
    y = torch.nn.functional.layer_norm(tx, (d,), tg, tb, 1e-5)
    np.testing.assert_allclose(O.layernorm(x, gamma, beta, 1e-5)[0], y.detach().numpy(), rtol=1e-11, atol=1e-11)
    (y * torch.tensor(dy)).sum().backward()
    dx, dg, db = O.layernorm_backward(dy, x, gamma, 1e-5, dres)
    for got, want in ((dx - dres, tx.grad), (dg, tg.grad), (db, tb.grad)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-9, atol=1e-10)
    # a central difference along a direction: error of order step^2, about 1e-8
    v, step = r.standard_normal((n, d)), 1e-4
    f = lambda z: (O.layernorm(z, gamma, beta, 1e-5)[0] * dy).sum()  # noqa: E731
    num = (f(x + step * v) - f(x - step * v)) / (2 * step)
    assert abs(num - ((dx - dres) * v).sum()) <= 1e-5 * (1 + abs(num))


def test_fp8_layer_without_rounding_is_the_plain_layer():
    # operands that E4M3 holds exactly: the FP8 forward's first product is the plain one
    r = np.random.default_rng(3)
    x = r.choice([-2.0, -1.0, 0.5, 1.0, 448.0], size=(6, 128)).astype(np.float32)
    x[:, 0] = 448.0
    np.testing.assert_array_equal(O.fp8_rows_value(x), x.astype(np.float64))
    w = r.standard_normal((128, 128))
    h = np.abs(r.standard_normal((6, 128)))
    np.testing.assert_allclose(O.fp8_rows_value(h), h, rtol=2.0 ** -4)
    y, a1, a3, hh = O.swiglu_expert_fp8b(x.astype(np.float64), w, w, np.eye(128))
    np.testing.assert_allclose(a1, x @ w.T, rtol=1e-12)
    np.testing.assert_array_equal(y, O.fp8_rows_value(hh))
