"""The draft side's operators as a user runs them together: a quantised head grows a draft tree
by beam selection with its states following their beams, the tree is pruned and verified, and
the target's outcome lists train the head's logits."""
import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv
import oracle
from oracle import draft_ops as ops

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


class Draft:
    """A small recurrent draft model: state' = tanh(state[parent] + embedding[token]), logits by a
    head whose weights were quantised once."""

    def __init__(self, D, V, seed):
        g = torch.Generator().manual_seed(seed)
        self.embed = torch.randn(V, D, generator=g).cuda()
        w = (torch.randn(V, D, generator=g) * 0.3).cuda()
        self.w, self.w_scale = torch.empty(V, D, dtype=torch.int8, device="cuda"), torch.empty(V, device="cuda")
        sv.spec_quantize_rows(w, self.w, self.w_scale)

    def logits(self, state, out):
        """state [rows, D] float32 -> out [rows, V] bf16 through the quantised product."""
        q = torch.empty(state.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(state.shape[0], device="cuda")
        sv.spec_quantize_rows(state, q, s)
        sv.spec_int8_product(q, s, self.w, self.w_scale, out)


def grow(model, B, W, D, V, depth):
    """A tree of depth * W nodes below the root for each sequence, level by level."""
    ctx = sv.spec_beam_init(B, W, W, V, torch.bfloat16)
    state = torch.zeros(1, B, W, D, device="cuda")
    root = torch.randint(0, V, (B,), generator=torch.Generator().manual_seed(1)).cuda()
    state[0] = torch.tanh(model.embed[root])[:, None, :]
    score = torch.full((B, W), -float("inf"), device="cuda")
    score[:, 0] = 0.0                                    # one beam to start from
    parent = torch.empty(B, W, dtype=torch.int32, device="cuda")
    token, logq = torch.empty_like(parent), torch.empty(B, W, device="cuda")
    logits = torch.empty(B, W, V, dtype=torch.bfloat16, device="cuda")
    levels = []
    for _ in range(depth):
        model.logits(state.view(B * W, D), logits.view(B * W, V))
        before, old = score.clone(), state.clone()
        sv.spec_beam_select(ctx, logits, score, None, parent, token, score, logq)
        sv.spec_beam_reorder(parent, state, state)
        levels.append(dict(logits=logits.float().cpu().numpy(), score=before.cpu().numpy(),
                           parent=parent.cpu().numpy(), token=token.cpu().numpy(), logq=logq.cpu().numpy(),
                           new=score.cpu().numpy(), old=old.cpu().numpy(), state=state.cpu().numpy()))
        state[0] = torch.tanh(state[0] + model.embed[token.long()])
    return root, levels


def test_a_tree_grown_pruned_and_verified():
    B, W, D, V, depth = 3, 4, 64, 3001, 3
    model = Draft(D, V, seed=2)
    root, levels = grow(model, B, W, D, V, depth)
    e = 2.0 ** -23 * (np.log(V) + 6)
    for lv in levels:
        p, t, v, q = ops.beam_select(lv["logits"], lv["score"], None, W)
        # tie borders aside (two values within 2 e), the order is the oracle's
        gaps = np.abs(np.diff(v, axis=1))
        assert (gaps > 2 * e).all(), "the seed gives two candidates that no rounding may order"
        assert np.array_equal(lv["parent"], p) and np.array_equal(lv["token"], t)
        assert (np.abs(lv["new"] - v) <= e + 2.0 ** -24 * np.abs(v)).all()
        assert np.array_equal(lv["state"], ops.beam_reorder(p, lv["old"], lv["old"]))
    # the levels as one tree in the layout that pruning and verification take
    M = 1 + depth * W
    parent = np.zeros((B, M), np.int32)
    token = np.zeros((B, M), np.int32)
    logq = np.zeros((B, M), np.float32)
    parent[:, 0] = -1                                    # the root
    for d, lv in enumerate(levels):
        at = slice(1 + d * W, 1 + (d + 1) * W)
        parent[:, at] = 0 if d == 0 else 1 + (d - 1) * W + lv["parent"]
        token[:, at], logq[:, at] = lv["token"], np.minimum(lv["logq"], 0)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    cum = torch.empty(B, M, dtype=torch.float64, device="cuda")
    new_index, new_parent = (torch.empty(B, M, dtype=torch.int32, device="cuda") for _ in range(2))
    count = torch.empty(B, dtype=torch.int32, device="cuda")
    sv.spec_tree_prune(dev(parent), dev(logq), -1e30, M, cum, new_index, new_parent, count)
    torch.cuda.synchronize()
    assert (count.cpu().numpy() == M).all()
    # a node's cumulative log-probability is the score its beam had: depth sums of binary32 values
    last = levels[-1]
    tol = depth * 2.0 ** -23 * np.abs(last["new"]) + depth * e
    assert (np.abs(cum.cpu().numpy()[:, -W:] - last["new"]) <= tol).all()
    # greedy verification against a target that follows the best path of the tree
    target = torch.zeros(B, M, V, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        path = [int(1 + (depth - 1) * W + np.argmax(last["new"][b]))]
        while path[-1] != 0:
            path.append(int(parent[b, path[-1]]))
        for x, child in zip(path[1:], path[:-1]):
            target[b, x, int(token[b, child])] = 5.0
    ctx = sv.spec_tree_verify_init(B, M, V, torch.bfloat16)
    length, extra = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    out = torch.empty(B, M, dtype=torch.int32, device="cuda")
    n_nodes = torch.full((B,), M, dtype=torch.int32, device="cuda")
    sv.spec_tree_verify_greedy(ctx, dev(parent), dev(token), n_nodes, target, length, out, extra)
    torch.cuda.synchronize()
    assert (length.cpu().numpy() == depth).all()
    ref = oracle.tree_verify_greedy(parent, token, np.full(B, M, np.int32), target.float().cpu().numpy())
    assert np.array_equal(ref["length"], length.cpu().numpy())


def test_outcome_lists_train_the_heads_logits():
    """The verifier's outcome lists (target row of the bonus position) as the teacher: steps against
    the gradient lower the loss's linear prediction, and the loss and gradient are the oracle's."""
    B, G, V, F = 4, 2, 5003, 16
    g = torch.Generator().manual_seed(7)
    draft = (torch.randn(B, G, V, generator=g) * 2).to(torch.bfloat16).cuda()
    target = (torch.randn(B, G + 1, V, generator=g) * 2).to(torch.bfloat16).cuda()
    tokens = torch.randint(0, V, (B, G), generator=g).int().cuda()
    temp = torch.ones(B, device="cuda")
    ctx = sv.spec_verify_init(B, G, V, torch.bfloat16)
    alen = torch.empty(B, dtype=torch.int32, device="cuda")
    toks = torch.empty(B, G + 1, dtype=torch.int32, device="cuda")
    sv.spec_verify(ctx, draft, target, tokens, temp, 0, 0, alen, toks)
    ids = torch.empty(B, G + 1, F, dtype=torch.int32, device="cuda")
    probs = torch.empty(B, G + 1, F, device="cuda")
    pk = torch.empty(B, G + 1, device="cuda")
    sv.spec_verify_outcomes(ctx, draft, target, tokens, F, ids, probs, pk)
    teach_ids = ids[:, G].contiguous()
    teacher = probs[:, G].log().contiguous()              # log-probabilities: normaliser 0
    tlse = torch.zeros(B, dtype=torch.float64, device="cuda")
    z = draft[:, G - 1].contiguous()
    weight = torch.full((B,), 1.0 / B, device="cuda")
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, dtype=torch.float64, device="cuda")
    grad = torch.empty(B, V, dtype=torch.bfloat16, device="cuda")
    sv.spec_distill_loss_grad(z, teach_ids, teacher, tlse, temp, weight, loss, lse, grad)
    torch.cuda.synchronize()
    ol, olse, og = ops.distill(z.float().cpu().numpy(), teach_ids.cpu().numpy(), teacher.cpu().numpy(),
                               tlse.cpu().numpy(), temp.cpu().numpy(), weight.cpu().numpy().astype(np.float64))
    e = 2.0 ** -23 * (np.log(V) + 6)
    assert (np.abs(loss.cpu().numpy() - ol) <= e + 2.0 ** -24 * np.abs(ol) + 1e-9).all()
    got = grad.float().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(og) * (1 + 2.0 ** -8) + np.abs(og) * 2.0 ** -16 + 2.0 ** -24 / B * e
    # listed entries are a difference of two terms: the tolerance counts both
    rows = np.arange(B)[:, None]
    tol[rows, teach_ids.cpu().numpy()] += e / B
    assert (np.abs(got - og) <= tol).all()
