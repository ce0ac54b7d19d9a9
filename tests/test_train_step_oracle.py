"""Pins of the oracle of the balance loss over sequences and of the backward from kept activations (CPU)."""
import numpy as np
import pytest
import torch

import oracle as O


def _case(n, e, k, seed):
    r = np.random.default_rng(seed)
    lg = r.standard_normal((n, e)) * 1.5
    return lg, np.argsort(-lg, axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_one_sequence_is_the_auxiliary_loss(gate):
    lg, idx = _case(50, 12, 3, 0)
    counts, loss, grad = O.balance_loss(lg, idx, [0, 50], gate, 0.01, 0.0)
    assert counts.sum() == 150
    assert loss[0] == pytest.approx(0.01 * O.aux_loss(lg, idx, 12, gate), rel=1e-12) and loss[1] == 0
    np.testing.assert_allclose(grad, 0.01 * O.aux_loss_grad(lg, idx, 12, gate), rtol=1e-10, atol=1e-16)


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_gradient_against_autograd(gate):
    """Both losses written again in torch operations, f fixed; padding rows and an empty sequence."""
    n, e, k, off = 40, 7, 2, [3, 3, 20, 31]
    lg, idx = _case(n, e, k, 1)
    counts, loss, grad = O.balance_loss(lg, idx, off, gate, 0.3, 0.05)
    t = torch.tensor(lg, requires_grad=True)
    q = torch.softmax(t, 1) if gate == "softmax" else torch.sigmoid(t) / torch.sigmoid(t).sum(1, keepdim=True)
    bal = sum(((torch.tensor(counts[s] / (off[s + 1] - off[s]))) * q[off[s]:off[s + 1]].mean(0)).sum()
              for s in (1, 2)) * 0.3 * e / 2
    z = 0.05 * (torch.logsumexp(t[3:31], 1) ** 2).mean()
    (bal + z).backward()
    np.testing.assert_allclose(loss, [bal.item(), z.item()], rtol=1e-12)
    np.testing.assert_allclose(grad, t.grad.numpy(), rtol=1e-9, atol=1e-15)
    assert not grad[:3].any() and not grad[31:].any() and not counts[0].any()


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_gradient_against_differences(gate):
    """A central difference of step 2^-12 is off by step^2 times a third derivative of order one."""
    n, e, off = 24, 6, [0, 10, 24]
    lg, idx = _case(n, e, 2, 2)
    counts, _, grad = O.balance_loss(lg, idx, off, gate, 1.0, 0.5)
    f = counts / np.diff(off)[:, None]
    v = np.random.default_rng(3).standard_normal((n, e))
    h = 2.0 ** -12
    up = O.balance_loss(lg + h * v, idx, off, gate, 1.0, 0.5, f)[1].sum()
    dn = O.balance_loss(lg - h * v, idx, off, gate, 1.0, 0.5, f)[1].sum()
    assert abs((up - dn) / (2 * h) - (grad * v).sum()) <= 1e-5


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_masked_experts_and_rows(gate):
    lg, idx = _case(6, 5, 2, 4)
    lg[1, 3] = -np.inf
    lg[2] = -np.inf
    counts, loss, grad = O.balance_loss(lg, idx, [0, 6], gate, 1.0, 1.0)
    assert np.isfinite(loss).all() and np.isfinite(grad).all()
    assert grad[1, 3] == 0 and not grad[2].any() and counts.sum() == 12


def test_swiglu_backward_against_autograd():
    r = np.random.default_rng(5)
    rows, d, f, off = 9, 4, 6, [0, 4, 4, 9]
    dy, w2 = r.standard_normal((rows, d)), r.standard_normal((3, d, f))
    a1, a3, g = r.standard_normal((rows, f)), r.standard_normal((rows, f)), r.random(rows)
    da1, da3, h, dg = O.swiglu_backward_kept(dy, off, w2, g, a1, a3)
    t1, t3, tg = (torch.tensor(v, requires_grad=True) for v in (a1, a3, g))
    act = torch.nn.functional.silu(t1) * t3
    y = torch.cat([act[a:b] @ torch.tensor(w2[i]).T for i, (a, b) in enumerate(zip(off, off[1:]))])
    ((tg[:, None] * y) * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(da1, t1.grad, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(da3, t3.grad, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dg, tg.grad, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(h, g[:, None] * act.detach().numpy(), rtol=1e-12)


def test_kept_values_invert_the_quantiser():
    """Half a step of E4M3 is 2^-4 of a value, or 2^-10 of the scale below its smallest normal number; a largest
    element above 448 scales (it lies below 512) is cut to 448."""
    r = np.random.default_rng(6)
    x = (r.standard_normal((5, 96)) * np.exp(3 * r.standard_normal((5, 96)))).astype(np.float32)
    codes, scales, _ = O.mx_quantize(x)
    v = O.kept_values(codes, scales.T)
    s = np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=1)
    assert (np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + np.maximum(np.abs(x) - 448 * s, 0)).all()
    np.testing.assert_array_equal(v.astype(np.float32), O.bf16_round(v))   # every value is a bf16 number
