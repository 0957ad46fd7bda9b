"""The 4-bit head and the token scores as a user runs them together: logits from quantised hidden
states and weights; the tokens' log-probabilities of draft and target into the accept test; the
normalisers into a beam selection; the target's lists as a teacher; the gradient back through the
head's weights."""
import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv
import oracle
from oracle import draft_ops as ops

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

U = 2.0 ** -24


class Head:
    """A head whose weights were quantised once."""

    def __init__(self, D, V, seed, other=None):
        """With `other`: weights that are correlated with that head's."""
        g = torch.Generator().manual_seed(seed)
        self.weight = (torch.randn(V, D, generator=g) * 0.2).cuda()
        if other is not None:
            self.weight = 0.9 * other.weight + 0.3 * self.weight
        whole = sv.spec_mxfp4_padded(D)
        self.w = torch.empty(V, whole // 2, dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(V, whole // 32, dtype=torch.uint8, device="cuda")
        self.values = torch.empty_like(self.weight)
        sv.spec_mxfp4_quantize_rows(self.weight, self.w, self.scale, self.values)

    def logits(self, hidden, dtype=torch.bfloat16):
        N, whole = hidden.shape[0], 2 * self.w.shape[1]
        q = torch.empty(N, whole // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(N, whole // 32, dtype=torch.uint8, device="cuda")
        values = torch.empty_like(hidden)
        sv.spec_mxfp4_quantize_rows(hidden, q, s, values)
        out = torch.empty(N, self.w.shape[0], dtype=dtype, device="cuda")
        sv.spec_mxfp4_product(q, s, self.w, self.scale, out)
        return out, values


class Scores:
    def __init__(self, logits, token, temperature, K):
        N, V = logits.shape
        self.ctx = sv.spec_logprobs_init(N, V, K, logits.dtype)
        f = lambda *s: torch.empty(*s, device="cuda")
        i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
        self.logprob, self.rank, self.entropy, self.norm = f(N), i(N), f(N), f(N, 2)
        self.top_token, self.top_logprob = (i(N, K), f(N, K)) if K else (None, None)
        sv.spec_token_logprobs(self.ctx, logits, token, temperature, self.logprob, self.rank, self.entropy,
                               self.top_token, self.top_logprob, self.norm)


def hidden(N, D, seed):
    return torch.randn(N, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def test_the_heads_logits_are_the_product_of_the_values():
    head = Head(500, 3001, 1)
    x = hidden(20, 500, 2)
    logits, values = head.logits(x, torch.float32)
    torch.cuda.synchronize()
    a, w = values.double().cpu().numpy(), head.values.double().cpu().numpy()
    want = a @ w.T
    # the header's bound, and the rounding of the output
    off = 512 / 64 * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T) + U * np.abs(want)
    assert (np.abs(logits.double().cpu().numpy() - want) <= off).all()


def test_scores_of_draft_and_target_into_the_accept_test():
    B, G, D, V = 6, 4, 200, 5003
    draft = Head(D, V, 3)
    target = Head(D, V, 4, draft)
    x = hidden(B * G, D, 5)
    zq, zp = draft.logits(x)[0], target.logits(x)[0]
    noise = torch.rand(B * G, V, generator=torch.Generator().manual_seed(6)).cuda()
    token = (zq.float() - torch.log(-torch.log(noise))).argmax(1).to(torch.int32)   # tokens drawn from the draft
    temperature = torch.ones(B * G, device="cuda")
    p, q = Scores(zp, token, temperature, 0), Scores(zq, token, temperature, 0)
    pairs = torch.stack((q.logprob, p.logprob), 1).view(B, G, 2).contiguous()
    ctx = sv.spec_verify_init(B, G, V, torch.bfloat16)
    length = torch.empty(B, dtype=torch.int32, device="cuda")
    sv.spec_accept_logprobs(ctx, pairs, 11, 0, length)
    # the whole verification of the same logits and uniforms keeps the same drafts
    bonus = target.logits(hidden(B, D, 7))[0]
    target_logits = torch.cat((zp.view(B, G, V), bonus[:, None]), 1).contiguous()
    full, tokens = torch.empty_like(length), torch.empty(B, G + 1, dtype=torch.int32, device="cuda")
    sv.spec_verify(ctx, zq.view(B, G, V), target_logits, token.view(B, G), torch.ones(B, device="cuda"), 11, 0, full, tokens)
    torch.cuda.synchronize()
    bf = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    ref = oracle.verify(bf(zq.view(B, G, V)), bf(target_logits), token.view(B, G).cpu().numpy(),
                        np.ones(B, np.float32), seed=11, offset=0)
    assert (np.abs(ref["acc_margin"][np.isfinite(ref["acc_margin"])]) > 1e-5).all(), "the seed gives a border"
    assert np.array_equal(length.cpu().numpy(), ref["accept_len"])
    assert np.array_equal(full.cpu().numpy(), ref["accept_len"])


def test_normalisers_into_the_beam_selection():
    B, W, K, D, V = 3, 4, 6, 128, 9001
    logits = Head(D, V, 8).logits(hidden(B * W, D, 9))[0]
    none = torch.full((B * W,), -1, dtype=torch.int32, device="cuda")
    s = Scores(logits, none, None, 20)
    lse = s.norm.double().sum(1).view(B, W).contiguous()
    score = -torch.rand(B, W, generator=torch.Generator().manual_seed(1)).cuda()
    ctx = sv.spec_beam_init(B, W, K, V, torch.bfloat16)
    parent, token = (torch.empty(B, K, dtype=torch.int32, device="cuda") for _ in range(2))
    value, logq = (torch.empty(B, K, device="cuda") for _ in range(2))
    sv.spec_beam_select(ctx, logits.view(B, W, V), score, lse, parent, token, value, logq)
    torch.cuda.synchronize()
    op, ot, ov, oq = ops.beam_select(logits.float().cpu().numpy().reshape(B, W, V), score.cpu().numpy(),
                                     lse.cpu().numpy(), K)
    assert np.array_equal(parent.cpu().numpy(), op) and np.array_equal(token.cpu().numpy(), ot)
    # every kept candidate is in its beam's list, with its log-probability (of the same normaliser,
    # rounded to binary32 twice on one way and once on the other)
    row = (torch.arange(B, device="cuda")[:, None] * W + parent).long().view(-1)
    found = s.top_token[row] == token.view(-1, 1)
    assert (found.sum(1) == 1).all()
    lp = s.top_logprob[row][found]
    off = U * (np.abs(oq.reshape(-1)) * 2 + 12) + 2.0 ** -23 * (np.log(V) + 6)
    assert (np.abs(lp.double().cpu().numpy() - oq.reshape(-1)) <= off).all()


@pytest.mark.parametrize("T", [1.0, 1.5])
def test_lists_as_a_teacher(T):
    """The target's lists with their log-probabilities, times T, as teacher logits and the teacher's
    normaliser 0: the distillation's loss is that of the target's own logits and normaliser."""
    N, D, V, K = 12, 256, 7001, 32
    x = hidden(N, D, 10)
    zq, zp = Head(D, V, 11).logits(x)[0], Head(D, V, 12).logits(x)[0]
    temperature = torch.full((N,), T, device="cuda")
    s = Scores(zp, torch.full((N,), -1, dtype=torch.int32, device="cuda"), temperature, K)
    zero = torch.zeros(N, dtype=torch.float64, device="cuda")
    weight = torch.full((N,), 1.0 / N, device="cuda")
    losses = []
    for teacher, lse in (((s.top_logprob * T).contiguous(), zero),
                         (zp.float().gather(1, s.top_token.long()).contiguous(), s.norm.double().sum(1).contiguous())):
        loss, norm = torch.empty(N, device="cuda"), torch.empty(N, dtype=torch.float64, device="cuda")
        grad = torch.empty_like(zq)
        sv.spec_distill_loss_grad(zq, s.top_token, teacher, lse, temperature, weight, loss, norm, grad)
        torch.cuda.synchronize()
        losses.append(loss.double().cpu().numpy())
        ol, _, _ = ops.distill(zq.float().cpu().numpy(), s.top_token.cpu().numpy(), teacher.cpu().numpy(),
                               lse.cpu().numpy(), temperature.cpu().numpy(), weight.cpu().numpy().astype(np.float64))
        e = 2.0 ** -23 * (np.log(V) + 6)
        assert (np.abs(losses[-1] - ol) <= e + U * np.abs(ol) + 1e-9).all()
    # teacher log-probabilities differ by their roundings (4 u |y| of |y| < 40, log S's u 10): relative
    # changes c of the p_j move the loss by sum p_j c (1 + |log p - log q|) at most
    c = U * (4 * 40 + 10) + 2.0 ** -23 * (np.log(V) + 6)
    assert (np.abs(losses[0] - losses[1]) <= c * (1 + 60)).all()


def test_a_training_step_through_the_heads_values():
    """Loss -sum_n a_n (logprob_n + b H_n) of the quantised head; its gradient for the weights, taken
    through their values, is the product of the logits' gradient with the hidden values."""
    N, D, V = 16, 96, 2003
    head = Head(D, V, 13)
    z, values = head.logits(hidden(N, D, 14), torch.float32)
    token = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(15)).to(torch.int32).cuda()
    temperature = torch.full((N,), 0.8, device="cuda")
    s = Scores(z, token, temperature, 0)
    a, b = torch.full((N,), -1.0 / N, device="cuda"), torch.full((N,), -0.01 / N, device="cuda")
    grad = torch.empty_like(z)
    sv.spec_token_logprobs_backward(s.ctx, z, token, temperature, s.norm, s.entropy, a, b, grad)
    torch.cuda.synchronize()
    want = ops.token_scores_grad(z.cpu().numpy(), token.cpu().numpy(), temperature.cpu().numpy(), a.cpu().numpy(), b.cpu().numpy())
    # relative parts of p and of the factor behind it, for log p and entropies below 32 in size
    off = 2.0 ** -23 * (np.log(V) + 6) + 40 * 2.0 ** -22
    got = grad.double().cpu().numpy()
    size = np.abs(want) + 1.25 * 1.32 / N * np.exp(ops.score_parts(z.double().cpu().numpy() * np.float32(1 / np.float32(0.8)))[0])
    assert (np.abs(got - want) <= off * size).all()
    step = grad.t().contiguous().double() @ values.double()                # [V, D]
    exact = want.T @ values.double().cpu().numpy()
    bound = (off * size).T @ np.abs(values.double().cpu().numpy())
    assert (np.abs(step.cpu().numpy() - exact) <= bound + 1e-12).all()


def test_the_chain_replayed_from_a_graph():
    N, D, V, K = 7, 160, 20011, 10
    head = Head(D, V, 16)
    x = hidden(N, D, 17)
    side = torch.cuda.Stream()
    whole = sv.spec_mxfp4_padded(D)
    q = torch.empty(N, whole // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(N, whole // 32, dtype=torch.uint8, device="cuda")
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    token = torch.arange(N, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    out = [f(N), i(N), f(N), i(N, K), f(N, K), f(N, 2)]
    a = torch.ones(N, device="cuda")
    ctx = sv.spec_logprobs_init(N, V, K, torch.bfloat16, stream=side)

    def step():
        sv.spec_mxfp4_quantize_rows(x, q, sc)
        sv.spec_mxfp4_product(q, sc, head.w, head.scale, z)
        sv.spec_token_logprobs(ctx, z, token, None, *out)
        sv.spec_token_logprobs_backward(ctx, z, token, None, out[5], out[2], a, a, z)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(3):
        x.copy_(hidden(N, D, 30 + n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        logits, _ = head.logits(x)
        s = Scores(logits, token, None, K)
        g = torch.empty_like(logits)
        sv.spec_token_logprobs_backward(s.ctx, logits, token, None, s.norm, s.entropy, a, a, g)
        torch.cuda.synchronize()
        for got, want in zip(out + [z], (s.logprob, s.rank, s.entropy, s.top_token, s.top_logprob, s.norm, g)):
            assert torch.equal(got, want)
