"""Beam selection that forms its own normalisers, with beams of large finite logits (masked with a
large constant throughout, in part, or with a few larger entries): log-probabilities against
(z - M) - log sum exp(z - M) with M the beam's largest logit, in 64 bits.

Tolerance as for ordinary beams: the normaliser's e = 2^-23 (ln V + 6) and the rounding of the
output to binary32; every pair of kept values of different beams is further apart than 2 e, so
parents and tokens are equal."""
import math

import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def reference(z, score, K):
    W, V = z.shape
    z = z.astype(np.float64)
    M = z.max(1, keepdims=True)
    logq = (z - M) - np.log(np.exp(z - M).sum(1, keepdims=True))
    value = score[:, None].astype(np.float64) + logq
    w, v = np.divmod(np.arange(W * V), V)
    order = np.lexsort((v, -z.ravel(), w, -value.ravel()))[:K]
    return w[order], v[order], value.ravel()[order], logq.ravel()[order]


@pytest.mark.parametrize("c", [-1e8, -1e10, -1e30, 1e30, "min", "max"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1003, 40009])
def test_beams_of_large_finite_logits(V, dtype, c):
    print(f"\n[beam far V={V} {dtype} {c}]", flush=True)
    info = torch.finfo(DTYPE[dtype])
    c = {"min": info.min, "max": info.max}.get(c, c)
    W, K = 5, 24
    g = torch.Generator().manual_seed(V)
    z = torch.randn(1, W, V, generator=g) * 2.5
    z[0, 0] = c                                       # masked throughout
    z[0, 1] = c if c < 0 else c * (1 - 2.0 ** -7)     # the same, five entries above the rest
    z[0, 1, torch.randperm(V, generator=g)[:5]] = c * (1 - 2.0 ** -7) if c < 0 else c
    z[0, 2, V // 4:] = c if c < 0 else -c             # ordinary entries in front
    z[0, 3, :V // 2] = c if c < 0 else -c             # and behind
    z = z.to(DTYPE[dtype])
    score = torch.tensor([[math.log(V) - 3.53, -1.01, -0.5, 0.0, -0.25]])
    ctx = sv.spec_beam_init(1, W, K, V, DTYPE[dtype])
    parent, token = (torch.empty(1, K, dtype=torch.int32, device="cuda") for _ in range(2))
    sc, lq = torch.empty(1, K, device="cuda"), torch.empty(1, K, device="cuda")
    sv.spec_beam_select(ctx, z.cuda(), score.cuda(), None, parent, token, sc, lq)
    torch.cuda.synchronize()
    w, v, value, logq = reference(z[0].float().numpy(), score[0].numpy(), K + 1)
    e = 2.0 ** -23 * (math.log(V) + 6)
    crossing = w[1:] != w[:-1]
    assert (np.abs(np.diff(value))[crossing] > 2 * e).all(), "two beams' values that no rounding may order"
    w, v, value, logq = w[:K], v[:K], value[:K], logq[:K]
    assert len(set(w)) >= 3
    assert np.array_equal(parent[0].cpu().numpy(), w) and np.array_equal(token[0].cpu().numpy(), v)
    assert (np.abs(sc[0].cpu().numpy() - value) <= e + 2.0 ** -24 * np.abs(value)).all()
    assert (np.abs(lq[0].cpu().numpy() - logq) <= e + 2.0 ** -24 * np.abs(logq)).all()
