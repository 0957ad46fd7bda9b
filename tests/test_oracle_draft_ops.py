"""Pins of the numpy forms of beam selection, state reordering, distillation, row
quantisation and the integer product (oracle/draft_ops.py), each by something other than
itself."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draft_ops as ops


def test_selection_is_the_sorted_order_of_the_tuples():
    rng = np.random.default_rng(3)
    for _ in range(20):
        B, W, V, K = 2, int(rng.integers(1, 5)), int(rng.integers(1, 12)), int(rng.integers(1, 9))
        z = rng.integers(-3, 4, (B, W, V)).astype(np.float32)
        z[rng.random(z.shape) < 0.1] = -np.inf
        score = -rng.integers(0, 3, (B, W)).astype(np.float32)
        score[rng.random(score.shape) < 0.2] = -np.inf
        lse = rng.integers(0, 3, (B, W)).astype(np.float64)
        p, t, val, q = ops.beam_select(z, score, lse, K)
        for b in range(B):
            cand = sorted((-(float(score[b, w]) + (float(z[b, w, v]) - lse[b, w])), w, -float(z[b, w, v]), v)
                          for w in range(W) for v in range(V)
                          if np.isfinite(z[b, w, v]) and np.isfinite(score[b, w]))[:K]
            for j in range(K):
                if j < len(cand):
                    assert (p[b, j], t[b, j], val[b, j]) == (cand[j][1], cand[j][3], -cand[j][0])
                else:
                    assert p[b, j] == -1 and t[b, j] == -1 and val[b, j] == -np.inf == q[b, j]


def test_selection_against_a_stable_sort_of_the_flat_values():
    rng = np.random.default_rng(4)
    z = rng.normal(0, 2, (3, 4, 50)).astype(np.float32)
    score = rng.normal(-3, 1, (3, 4)).astype(np.float32)
    p, t, val, q = ops.beam_select(z, score, None, 6)
    lp = torch.log_softmax(torch.from_numpy(z).double(), -1)
    flat = (lp + torch.from_numpy(score).double()[..., None]).flatten(1)
    v, i = flat.sort(dim=1, descending=True, stable=True)
    assert np.array_equal((i[:, :6] // 50).numpy(), p) and np.array_equal((i[:, :6] % 50).numpy(), t)
    np.testing.assert_allclose(val, v[:, :6].numpy(), rtol=0, atol=1e-13)


def test_reorder_against_indexing():
    rng = np.random.default_rng(5)
    src, dst = rng.normal(size=(2, 3, 4, 5)), rng.normal(size=(2, 3, 6, 5))
    parent = rng.integers(-1, 5, (3, 6)).astype(np.int32)  # 4 lies outside, too
    out = ops.beam_reorder(parent, src, dst)
    keep = (parent < 0) | (parent >= 4)
    want = np.take_along_axis(src, np.where(keep, 0, parent)[None, :, :, None], axis=2)
    assert np.array_equal(out, np.where(keep[None, :, :, None], dst, want))


@pytest.mark.parametrize("full", [False, True])
def test_loss_and_gradient_against_autograd(full):
    rng = np.random.default_rng(6)
    N, V, K = 5, 23, 7
    z = torch.from_numpy(rng.normal(0, 2, (N, V))).requires_grad_()
    ids = rng.integers(0, V, (N, K)).astype(np.int32)   # with repetitions
    ids[0, 3:] = -1
    y = rng.normal(0, 2, (N, K))
    tl = rng.normal(4, 0.1, N) if full else None
    weight, r = rng.normal(size=N), np.ones(N)
    loss, lse, grad = ops.distill_scaled(z.detach().numpy(), ids, y, tl, weight, r)
    yt = torch.from_numpy(np.where(ids >= 0, y, -np.inf))
    logp = yt - torch.from_numpy(tl)[:, None] if full else torch.log_softmax(yt, 1)
    used = torch.from_numpy(ids >= 0)
    logq = torch.log_softmax(z, 1).gather(1, torch.from_numpy(np.maximum(ids, 0)).long())
    want = torch.where(used, logp.exp() * (torch.where(used, logp, 0.0) - logq), 0.0).sum(1)
    (want * torch.from_numpy(weight)).sum().backward()
    np.testing.assert_allclose(loss, want.detach().numpy(), rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(z, 1).detach().numpy(), rtol=0, atol=1e-12)
    np.testing.assert_allclose(grad, z.grad.numpy(), rtol=0, atol=1e-12)


def test_gradient_against_central_differences():
    rng = np.random.default_rng(7)
    N, V, K, h = 2, 9, 4, 1e-5
    x = rng.normal(0, 1, (N, V))
    ids = np.array([[1, 5, 5, -1], [0, 2, 3, 8]], np.int32)
    y = rng.normal(0, 1, (N, K))
    weight, r = np.array([0.5, 2.0]), np.ones(N)
    _, _, grad = ops.distill_scaled(x, ids, y, None, weight, r)
    for n in range(N):
        for v in range(V):
            up, down = x.copy(), x.copy()
            up[n, v] += h
            down[n, v] -= h
            d = (ops.distill_scaled(up, ids, y, None, weight, r)[0][n] -
                 ops.distill_scaled(down, ids, y, None, weight, r)[0][n]) / (2 * h)
            # the third derivative of a log-sum-exp is below 1: h^2 plus the rounding of the difference
            assert abs(weight[n] * d - grad[n, v]) < 2 * (h * h + 1e-10)


def test_distill_sentinels():
    z = np.zeros((7, 4), np.float32)
    z[3] = -np.inf
    z[5, 1] = np.nan
    ids = np.array([[-1, -1], [0, 4], [0, 1], [0, 1], [2, 3], [0, 1], [0, 1]], np.int32)
    teacher = np.zeros((7, 2), np.float32)
    teacher[4] = -np.inf
    temp = np.array([0.0, 1, 0.0, 1, 1, 1, 2], np.float32)
    loss, lse, grad = ops.distill(z, ids, teacher, None, temp, np.ones(7))
    assert loss[0] == 0 and (grad[0] == 0).all() and np.isnan(lse[0])      # no entry
    for n in (1, 2, 3, 5):                                                  # id, T, no logit, NaN
        assert np.isnan(loss[n]) and np.isnan(lse[n]) and np.isnan(grad[n]).all()
    assert loss[4] == 0 and (grad[4] == 0).all()                            # no teacher mass
    assert abs(loss[6] - np.log(2)) < 1e-12                                 # log 4 - log 2
    np.testing.assert_allclose(grad[6], 0.5 * (0.25 - np.array([0.5, 0.5, 0, 0])), atol=1e-15)


def test_quantisation_against_exact_fractions():
    rng = np.random.default_rng(8)
    x = rng.normal(0, 1, (4, 40)).astype(np.float32)
    x[1] = np.round(x[1] * 4) / 4
    x[1, 0] = 31.75                       # scale 0.25: exact ties at odd multiples of 0.125
    x[1, 1:9] = np.array([0.125, 0.375, -0.125, -0.375, 0.625, 5.125, -5.375, 31.625], np.float32)
    x[2] = 0
    q, scale = ops.quantize_rows(x)
    assert scale[2] == 0 and not q[2].any()
    for n in (0, 1, 3):
        s = Fraction(float(scale[n]))
        assert scale[n] == np.float32(np.abs(x[n]).max()) / np.float32(127)
        for k in range(x.shape[1]):
            assert q[n, k] == max(-127, min(127, round(Fraction(float(x[n, k])) / s)))  # ties to even
    x[3, 5] = np.inf
    q, scale = ops.quantize_rows(x)
    assert np.isnan(scale[3]) and not q[3].any()


def test_product_against_python_integers():
    rng = np.random.default_rng(9)
    a, w = (rng.integers(-128, 128, s).astype(np.int8) for s in ((3, 16), (5, 16)))
    sa, sw = rng.random(3).astype(np.float32), rng.random(5).astype(np.float32)
    out = ops.int8_product(a, sa, w, sw)
    for n in range(3):
        for v in range(5):
            acc = sum(int(x) * int(y) for x, y in zip(a[n], w[v]))
            assert out[n, v] == np.float32(np.float32(np.float32(acc) * sa[n]) * sw[v])
