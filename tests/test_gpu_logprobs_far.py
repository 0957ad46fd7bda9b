"""The gradient of the token scores at entries far below the others: their probabilities are less than
binary32's normal numbers, the gradients of large weights are not.

Bounds as in tests/test_gpu_logprobs.py, with u = 2^-24: at an entry of log-probability l the kernel's
p is off by P = D + u log S + 2^-22 (1 + |l|) of itself, l by P, H by E + u H, three more products and
sums 3 u; half a step of the type, which below the normal numbers is half of its smallest number."""
import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv
from oracle import draft_ops as ops

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def gradient(z, token, temperature, a, b):
    N, V = z.shape
    ctx = sv.spec_logprobs_init(N, V, 0, z.dtype)
    f = lambda *s: torch.full(s, 7.0, device="cuda")
    logprob, entropy, norm, grad = f(N), f(N), f(N, 2), torch.full_like(z, 7.0)
    rank = torch.empty(N, dtype=torch.int32, device="cuda")
    sv.spec_token_logprobs(ctx, z, token, temperature, logprob, rank, entropy, None, None, norm)
    sv.spec_token_logprobs_backward(ctx, z, token, temperature, norm, entropy, a, b, grad)
    torch.cuda.synchronize()
    return grad.double().cpu().numpy()


def check(z, token, temperature, a, b):
    got = gradient(z, token, temperature, a, b)
    zf, token, a, b = z.float().cpu().numpy(), token.cpu().numpy(), a.cpu().numpy(), b.cpu().numpy()
    temperature = None if temperature is None else temperature.cpu().numpy()
    x, r = ops.score_scaled(zf, temperature)
    l, p, h = ops.score_parts(x)
    _, log_s = ops.row_parts(x)
    want = ops.token_scores_grad(zf, token, temperature, a, b)
    d = np.where(p > 0, np.abs(x.astype(np.float64) - x.max(1).astype(np.float64)[:, None]), 0.0)
    mean = (p * d).sum(1)[:, None]
    D = 2.0 ** -23 * (np.log(z.shape[1]) + 6)
    E = (p * 2.0 ** -22 * (1 + d) * (1 + d + mean)).sum(1)[:, None] + 4 * U * mean
    al = np.where(p > 0, np.abs(l), 0.0)
    P = D + U * np.abs(log_s)[:, None] + 2.0 ** -22 * (1 + al)
    a64, b64 = np.abs(a.astype(np.float64))[:, None], np.abs(b.astype(np.float64))[:, None]
    size = a64 + b64 * (al + h[:, None])
    off = p * (size * (P + 3 * U) + b64 * (P + E + U * h[:, None])) * r[:, None]
    half, least = (U, 2.0 ** -149) if z.dtype == torch.float32 else (2.0 ** -8, 2.0 ** -133)
    # bf16 is rounded to by way of binary32
    off = off + half * (np.abs(want) + off) + least / 2 + (2.0 ** -150 if least > 2.0 ** -149 else 0)
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], off[bad][:5])
    return got, want


def rows(N, V, depth):
    """Rows whose first entries lie together and whose others go down to `depth` below them."""
    g = torch.Generator().manual_seed(int(depth))
    z = torch.randn(N, V, generator=g)
    z[:, 40:] = -torch.rand(N, V - 40, generator=g) * depth
    z[:, 5::97] = -float("inf")
    return z, torch.randint(0, 40, (N,), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("weight", [1e-10, 1.0, 1e10, 9e24, 1.1e25, 1e27, 1e30, 3e34])
def test_entries_below_the_normal_numbers(weight, dtype):
    N, V = 6, 3003
    z, token = rows(N, V, 190.0)
    z = z.to(DTYPE[dtype]).cuda()
    a = torch.tensor([1.0, -1.0, 0.0, 0.5, 1.0, 0.0], device="cuda") * weight
    b = torch.tensor([0.0, 0.5, 1.0, -1.0, 0.25, -0.5], device="cuda") * weight
    got, want = check(z, token, None, a, b)
    if 1e10 <= weight:           # some entries' p is subnormal, and their gradient an ordinary number
        _, p, _ = ops.score_parts(z.float().cpu().numpy())
        deep = (p > 0) & (p < 2.0 ** -127) & (np.abs(want) > 2.0 ** -125)
        assert deep.any() and (got[deep] != 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1e-30, 1e-3, 0.02])
def test_low_temperatures(T, dtype):
    """One entry has nearly all of the probability; at 1e-30 the others have none."""
    N, V = 6, 3001
    z, token = rows(N, V, 3.0)
    z = z.to(DTYPE[dtype]).cuda()
    g = torch.Generator().manual_seed(3)
    a, b = (torch.randn(N, generator=g).cuda() * 1e-8 for _ in range(2))
    check(z, token, torch.full((N,), T, device="cuda"), a, b)
