"""Pins of the scores' gradient at masked entries (oracle/draft_ops.py), on the CPU."""
import numpy as np
import torch

from oracle import draft_ops as ops


def test_a_masked_token_has_the_gradient_of_the_formula():
    """r a at the token itself (p = 0 there), 0 at the other masked entries, and nothing at all in a
    row that has only masked entries: autograd's, of the same logarithm."""
    z = np.array([[1.0, -np.inf, 0.5, -np.inf], [-np.inf] * 4], np.float32)
    token, a, b = np.array([1, 1], np.int32), np.array([0.75, 0.75], np.float32), np.array([-0.5, -0.5], np.float32)
    temperature = np.array([2.0, 2.0], np.float32)
    got = ops.token_scores(z, token, temperature, 0)
    assert got["logprob"].tolist() == [-np.inf, -np.inf] and got["rank"].tolist() == [2, -1]
    g = ops.token_scores_grad(z, token, temperature, a, b)
    assert g[0, 1] == 0.5 * 0.75 and g[0, 3] == 0 and (g[1] == 0).all()
    x = torch.tensor(z[:1] / 2).double().requires_grad_()
    torch.log_softmax(x, 1)[0, 1].backward()
    assert x.grad[0, 1] == 1 and x.grad[0, 3] == 0


def test_masked_entries_have_no_gradient_whatever_the_weights():
    z = np.array([[1.0, -np.inf, 0.5]] * 3, np.float32)
    token = np.array([0, 0, -1], np.int32)
    a, b = np.array([np.inf, 1, np.nan], np.float32), np.array([0, np.nan, 1], np.float32)
    with np.errstate(invalid="ignore"):
        g = ops.token_scores_grad(z, token, None, a, b)
    assert (g[:, 1] == 0).all() and not np.isfinite(g[:2, [0, 2]]).any() and np.isfinite(g[2]).all()
