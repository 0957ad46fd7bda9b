"""Pins of the oracle's 4-bit forms and token scores (oracle/draft_ops.py), on the CPU."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draft_ops as ops

LEVELS = [Fraction(v) for v in (0, Fraction(1, 2), 1, Fraction(3, 2), 2, 3, 4, 6)]


def nearest(y):
    """The code of |y| (a Fraction): the nearest level, ties to the even code, at most 6."""
    best = min(range(8), key=lambda c: (abs(LEVELS[c] - y), c % 2))
    return best


def test_quantisation_by_exact_fractions():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 75)) * np.exp(rng.standard_normal((6, 1)) * 8)).astype(np.float32)
    x[1, :32] = 0
    x[2, 3] = 1e-40                                   # a block with subnormal entries
    x[2, 32:64] = np.linspace(-3e-39, 3e-39, 32)
    x[3, :32] = np.float32(3.4e38) * np.linspace(-1, 1, 32).astype(np.float32)
    x[4, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0]
    x[4, 16:32] = 0.1
    q, scale, values = ops.mxfp4_quantize(x)
    assert q.shape == (6, 64) and scale.shape == (6, 4)
    for n in range(6):
        for b in range(4):
            block = [Fraction(float(v)) for v in x[n, 32 * b:32 * b + 32]]
            top = max([abs(v) for v in block], default=Fraction(0))
            e = -127
            while top >= Fraction(2) ** (e + 3):      # e = floor(log2 top) - 2
                e += 1
            assert scale[n, b] == e + 127
            for i in range(32):
                k = 32 * b + i
                code = (q[n, k // 2] >> (4 * (k % 2))) & 15
                want = nearest(abs(block[i]) / Fraction(2) ** e) if i < len(block) else 0
                assert code & 7 == want
                if i < len(block):
                    assert bool(code & 8) == bool(np.signbit(x[n, k]))
                    assert Fraction(float(values[n, k])) == (-1 if code & 8 else 1) * LEVELS[want] * Fraction(2) ** e
                else:
                    assert code == 0
    assert np.array_equal(ops.mxfp4_values(q, scale)[:, :75], values)


def test_quantisation_of_a_block_with_nan():
    x = np.ones((2, 64), np.float32)
    x[0, 3], x[1, 40] = np.nan, -np.inf
    q, scale, values = ops.mxfp4_quantize(x)
    assert scale.tolist() == [[255, 125, 0, 0], [125, 255, 0, 0]]
    assert np.isnan(values[0, :32]).all() and (values[0, 32:] == 1).all()
    assert np.isnan(ops.mxfp4_values(q, scale)[1, 32:64]).all()


def test_product_by_exact_fractions():
    rng = np.random.default_rng(1)
    q, w = rng.integers(0, 256, (3, 64)).astype(np.uint8), rng.integers(0, 256, (4, 64)).astype(np.uint8)
    s, t = rng.integers(100, 150, (3, 4)).astype(np.uint8), rng.integers(100, 150, (4, 4)).astype(np.uint8)
    out, size = ops.mxfp4_product(q, s, w, t)
    code = lambda row, k: int(row[k // 2] >> (4 * (k % 2))) & 15
    value = lambda c: (-1 if c & 8 else 1) * LEVELS[c & 7]
    for n in range(3):
        for v in range(4):
            terms = [value(code(q[n], k)) * value(code(w[v], k)) *
                     Fraction(2) ** (int(s[n, k // 32]) + int(t[v, k // 32]) - 254) for k in range(128)]
            assert abs(Fraction(float(out[n, v])) - sum(terms)) <= Fraction(float(size[n, v])) * 128 * Fraction(2) ** -53
            assert abs(Fraction(float(size[n, v])) - sum(map(abs, terms))) <= sum(map(abs, terms)) * 128 * Fraction(2) ** -53


def rows(N=9, V=40, seed=2):
    rng = np.random.default_rng(seed)
    z = np.round(rng.standard_normal((N, V)) * 3, 1).astype(np.float32)       # ties
    z[rng.random((N, V)) < 0.2] = -np.inf
    token = rng.integers(0, V, N).astype(np.int32)
    token[3] = -1
    return z, token, rng.uniform(0.5, 2, N).astype(np.float32)


def test_scores_by_sorting_and_log_softmax():
    z, token, temperature = rows()
    got = ops.token_scores(z, token, temperature, 7)
    x, r = ops.score_scaled(z, temperature)
    logp = torch.log_softmax(torch.from_numpy(x).double(), 1)
    h = torch.special.entr(logp.exp()).sum(1).numpy()
    for n in range(len(z)):
        order = sorted(range(z.shape[1]), key=lambda v: (-z[n, v], v))
        if token[n] >= 0:
            assert got["rank"][n] == order.index(token[n])
            np.testing.assert_allclose(got["logprob"][n], logp[n, token[n]], rtol=1e-12)
        else:
            assert got["rank"][n] == -1 and got["logprob"][n] == 0
        assert got["top_token"][n].tolist() == order[:7]
        np.testing.assert_allclose(got["top_logprob"][n], logp[n, order[:7]].numpy(), rtol=1e-12)
    np.testing.assert_allclose(got["entropy"], h, rtol=1e-12)
    np.testing.assert_allclose(got["norm"].sum(1), torch.logsumexp(torch.from_numpy(x).double(), 1).numpy(), rtol=1e-12)


def test_scores_of_empty_and_bad_rows():
    z = np.zeros((6, 5), np.float32)
    z[0] = -np.inf
    z[1, 2], z[2, 2] = np.nan, np.inf
    z[3, 1:] = -np.inf
    token = np.array([1, 1, 1, 2, 5, -1], np.int32)
    got = ops.token_scores(z, token, None, 3)
    assert got["logprob"][0] == -np.inf and got["norm"][0].tolist() == [-np.inf, 0] and got["rank"][0] == -1
    assert got["entropy"][0] == 0 and (got["top_token"][0] == -1).all() and (got["top_logprob"][0] == -np.inf).all()
    for n in (1, 2):
        assert np.isnan(got["logprob"][n]) and np.isnan(got["entropy"][n]) and np.isnan(got["top_logprob"][n]).all()
        assert got["rank"][n] == -1 and (got["top_token"][n] == -1).all()
    assert got["logprob"][3] == -np.inf and got["rank"][3] == 2 and got["top_token"][3].tolist() == [0, -1, -1]
    assert np.isnan(got["logprob"][4]) and got["rank"][4] == -1 and got["top_token"][4].tolist() == [0, 1, 2]
    assert got["logprob"][5] == 0 and got["rank"][5] == -1
    t = np.array([0, -1, np.inf, np.nan, 1e-45, 1], np.float32)
    bad = ops.token_scores(np.zeros((6, 5), np.float32), np.zeros(6, np.int32), t, 1)
    assert np.isnan(bad["logprob"][:5]).all() and np.isfinite(bad["logprob"][5])


def test_gradient_by_autograd_and_differences():
    z, token, temperature = rows(seed=3)
    rng = np.random.default_rng(4)
    a, b = rng.standard_normal(len(z)).astype(np.float32), rng.standard_normal(len(z)).astype(np.float32)
    got = ops.token_scores_grad(z, token, temperature, a, b)
    x, r = ops.score_scaled(z, temperature)
    xt = torch.from_numpy(np.where(np.isinf(x), -1e9, x)).double().requires_grad_()   # exp is 0 all the same
    logp = torch.log_softmax(xt, 1)
    given = torch.from_numpy(token) >= 0
    lp = logp.gather(1, torch.from_numpy(token).long().clamp(min=0)[:, None])[:, 0] * given
    loss = (torch.from_numpy(a).double() * lp + torch.from_numpy(b).double() * -(logp.exp() * logp).sum(1)).sum()
    loss.backward()
    np.testing.assert_allclose(got, xt.grad.numpy() * r[:, None].astype(np.float64), rtol=1e-9, atol=1e-12)

    def value(x):
        l, p, h = ops.score_parts(x)
        picked = np.where(token >= 0, l[np.arange(len(l)), np.maximum(token, 0)], 0.0)
        return a.astype(np.float64) * picked + b.astype(np.float64) * h

    x = rng.standard_normal(z.shape)
    g = ops.score_grad_scaled(x, token, a.astype(np.float64), b.astype(np.float64), np.ones(len(z)))
    step = 1e-5
    for v in range(0, z.shape[1], 7):
        up, down = x.copy(), x.copy()
        up[:, v] += step
        down[:, v] -= step
        np.testing.assert_allclose((value(up) - value(down)) / (2 * step), g[:, v], rtol=1e-6, atol=1e-8)


def test_gradient_of_empty_and_bad_rows():
    z = np.zeros((5, 4), np.float32)
    z[0] = -np.inf
    z[1, 0] = np.nan
    token = np.array([1, 1, 4, -1, 2], np.int32)
    g = ops.token_scores_grad(z, token, np.array([1, 1, 1, 1, 0], np.float32), np.ones(5, np.float32), None)
    assert (g[0] == 0).all() and np.isnan(g[1]).all() and np.isnan(g[2]).all() and np.isnan(g[4]).all()
    assert (g[3] == 0).all()


@pytest.mark.parametrize("shift", [1e4, 1e9, -1e30])
def test_scores_do_not_lose_the_sum_of_far_rows(shift):
    z = np.full((1, 8), shift, np.float32)
    got = ops.token_scores(z, np.array([3], np.int32), None, 1)
    np.testing.assert_allclose(got["logprob"], -np.log(8), rtol=1e-15)
    np.testing.assert_allclose(got["entropy"], np.log(8), rtol=1e-15)
