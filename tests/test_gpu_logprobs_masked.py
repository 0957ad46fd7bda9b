"""The gradient of the token scores at masked entries, on the GPU."""
import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


def score_and_gradient(z, token, temperature, a, b):
    N, V = z.shape
    ctx = sv.spec_logprobs_init(N, V, 0, z.dtype)
    f = lambda *s: torch.full(s, 7.0, device="cuda")
    logprob, entropy, norm = f(N), f(N), f(N, 2)
    rank = torch.empty(N, dtype=torch.int32, device="cuda")
    sv.spec_token_logprobs(ctx, z, token, temperature, logprob, rank, entropy, None, None, norm)
    grad = torch.full_like(z, 7.0)
    sv.spec_token_logprobs_backward(ctx, z, token, temperature, norm, entropy, a, b, grad)
    torch.cuda.synchronize()
    return logprob, rank, grad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [13, 9001])
def test_a_masked_token_has_the_gradient_of_the_formula(V, dtype):
    """r a at the token itself, wherever it lies, exactly; 0 at the other masked entries."""
    g = torch.Generator().manual_seed(V)
    N = 8
    z = torch.randn(N, V, generator=g)
    token = torch.tensor([0, 1, V - 1, V - 2, 5, 7, V // 2, 3], dtype=torch.int32)
    z[torch.rand(N, V, generator=g) < 0.4] = -INF
    z[:, 2] = 1.0
    z[torch.arange(N), token.long()] = -INF
    z[7] = -INF                                       # nothing but masked entries
    masked = torch.isinf(z).cuda()
    z, token = z.to(DTYPE[dtype]).cuda(), token.cuda()
    temperature, a = torch.full((N,), 2.0, device="cuda"), torch.full((N,), 0.75, device="cuda")
    logprob, rank, grad = score_and_gradient(z, token, temperature, a, -a)
    assert (logprob == -INF).all() and (rank[:7] >= 0).all() and rank[7] == -1
    want = torch.zeros_like(grad)
    want[torch.arange(N), token.long()] = 0.5 * 0.75
    want[7] = 0
    assert torch.equal(grad[masked], want[masked])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_entries_of_rows_with_weights_that_are_not_finite(dtype):
    """0 as ever, though nothing times such a weight is NaN; the row's other entries are not finite."""
    inf, nan = float("inf"), float("nan")
    N, V = 6, 9001
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(1))
    z[:, 100:4000] = z[:, V - 3:] = -INF
    z = z.to(DTYPE[dtype]).cuda()
    masked = torch.isinf(z)
    token = torch.tensor([5, 5, 5, 5, 200, -1], dtype=torch.int32, device="cuda")
    a = torch.tensor([inf, nan, 1.0, -inf, nan, inf], device="cuda")
    b = torch.tensor([0.0, 1.0, nan, inf, 0.0, 0.5], device="cuda")
    grad = score_and_gradient(z, token, None, a, b)[2]
    masked[4, 200] = False                            # the token itself: r a
    assert torch.isnan(grad[4, 200])
    assert (grad[masked] == 0).all()
    assert not torch.isfinite(grad[:5][~masked[:5]]).any() and torch.isfinite(grad[5]).all()
