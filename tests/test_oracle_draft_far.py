"""The draft operators' oracle on rows of large finite logits: shifting a row by a constant changes
neither its distribution nor its loss, however large the constant."""
import numpy as np
import pytest

from oracle import draft_ops as ops


@pytest.mark.parametrize("shift", [2.0 ** 26, -2.0 ** 33, 2.0 ** 100, -2.0 ** 127])
def test_distillation_of_shifted_rows(shift):
    rng = np.random.default_rng(3)
    N, V, K = 5, 300, 4
    # two values of a row, so that the shifted ones are exact: shift, and shift less one step of it
    step = abs(shift) * 2.0 ** -20
    low = rng.random((N, V)) < 0.4
    x = np.where(low, -step, 0.0)
    ids = rng.integers(0, V, (N, K)).astype(np.int32)
    y, weight, r = rng.standard_normal((N, K)), rng.standard_normal(N), np.ones(N)
    loss, lse, grad = ops.distill_scaled(x, ids, y, None, weight, r)
    far_loss, far_lse, far_grad = ops.distill_scaled(x + shift, ids, y, None, weight, r)
    assert np.allclose(far_loss, loss, rtol=1e-13, atol=1e-13) and np.allclose(far_grad, grad, rtol=1e-13, atol=1e-15)
    assert np.allclose(far_lse, lse + shift, rtol=2.0 ** -52)
    assert np.allclose(grad.sum(1), 0, atol=1e-12)


@pytest.mark.parametrize("shift", [2.0 ** 26, -2.0 ** 100])
def test_selection_of_a_shifted_beam(shift):
    V = 50
    z = np.full((1, 2, V), np.float32(shift), np.float32)
    z[0, 1] = np.linspace(-2, 2, V)
    score = np.zeros((1, 2), np.float32)
    parent, token, value, logq = ops.beam_select(z, score, None, V + 3)
    q = logq[parent == 0]
    assert q.size and np.allclose(q, -np.log(V), rtol=1e-14)
    assert np.all(np.diff(value[0]) <= 0)
