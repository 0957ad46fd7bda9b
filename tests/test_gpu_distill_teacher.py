"""The verifier's outcome lists as a teacher: which of them is the target's row, and a step against
the gradient that they give."""
import math

import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

B, G, V, F = 4, 2, 5003, 16


def outcome_lists():
    g = torch.Generator().manual_seed(11)
    draft = (torch.randn(B, G, V, generator=g) * 2).to(torch.bfloat16).cuda()
    target = (torch.randn(B, G + 1, V, generator=g) * 2).to(torch.bfloat16).cuda()
    tokens = torch.randint(0, V, (B, G), generator=g).int().cuda()
    ctx = sv.spec_verify_init(B, G, V, torch.bfloat16)
    sv.spec_verify(ctx, draft, target, tokens, torch.ones(B, device="cuda"), 0, 0,
                   torch.empty(B, dtype=torch.int32, device="cuda"),
                   torch.empty(B, G + 1, dtype=torch.int32, device="cuda"))
    ids = torch.empty(B, G + 1, F, dtype=torch.int32, device="cuda")
    probs = torch.empty(B, G + 1, F, device="cuda")
    sv.spec_verify_outcomes(ctx, draft, target, tokens, F, ids, probs, torch.empty(B, G + 1, device="cuda"))
    torch.cuda.synchronize()
    return draft, target, ids, probs


def test_only_the_last_list_is_the_targets_row():
    draft, target, ids, probs = outcome_lists()
    p = torch.softmax(target.double(), -1)
    at = torch.gather(p, 2, ids.long())
    # "a relative error of a few 1e-6" of the lists' probabilities
    assert ((probs[:, G] - at[:, G]).abs() <= 1e-5 * at[:, G]).all()
    residual = (p[:, :G] - torch.softmax(draft.double(), -1)).clamp(min=0)
    want = torch.gather(residual / residual.sum(-1, keepdim=True), 2, ids[:, :G].long())
    assert ((probs[:, :G] - want).abs() <= 1e-5 * want + 1e-7).all()
    assert ((probs[:, :G] - at[:, :G]).abs() > 1e-2 * at[:, :G]).any(-1).all()   # another distribution


def test_a_step_against_the_gradient_lowers_the_loss_by_its_square():
    """f(z - h grad) = f(z) - h |grad|^2 + R with 0 <= R <= h^2 / 2 * |grad|^2 * L: the Hessian of a
    row's weight * loss is weight * P (diag q - q q^T), whose eigenvalues are at most weight * P / 2."""
    draft, _, ids, probs = outcome_lists()
    z = draft[:, G - 1].float().contiguous()
    ids, teacher = ids[:, G].contiguous(), probs[:, G].log().contiguous()
    zero, one = torch.zeros(B, dtype=torch.float64, device="cuda"), torch.ones(B, device="cuda")
    weight = torch.full((B,), 1.0 / B, device="cuda")
    loss, lse, grad = torch.empty(B, device="cuda"), zero.clone(), torch.empty_like(z)
    sv.spec_distill_loss_grad(z, ids, teacher, zero, one, weight, loss, lse, grad)
    h = 0.5
    after = torch.empty(B, device="cuda")
    sv.spec_distill_forward((z - h * grad).contiguous(), ids, teacher, zero, one, after, lse)
    torch.cuda.synchronize()
    square = grad.double().square().sum().item()
    drop = ((loss.double() - after.double()) * weight).sum().item()
    P = probs[:, G].double().sum(-1).max().item()
    # two losses a row, each within 2^-23 (ln V + 6) and half a step; z - h grad is rounded once,
    # which moves the loss by at most |grad| 2^-24 |z| in every entry
    err = 2 * (2.0 ** -23 * (math.log(V) + 6) + 2.0 ** -24 * loss.max().item())
    err += (grad.double().abs() * z.double().abs()).sum().item() * 2.0 ** -24
    # the gradient's own error is far below its square's second-order share
    room = h * h / 2 * square * P / 2 / B + 1e-5 * h * square
    assert square > 100 * err
    assert -room - err <= drop - h * square <= 1e-5 * h * square + err
