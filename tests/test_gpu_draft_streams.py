"""The selection and the reordering that follows it, on streams other than the one the context was
made with."""
import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def test_a_context_moved_to_the_current_stream():
    """Selection and in-place reordering stay in order on each stream that the context is moved to,
    however long the selection takes (a large one, so that an early reordering would read the old
    parents)."""
    B, W, V, S = 32, 16, 100003, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.empty(B, W, V, dtype=torch.bfloat16, device="cuda").normal_(0, 2.5, generator=g)
    start = torch.randint(0, 1 << 20, (2, B, W, S), dtype=torch.int32, device="cuda", generator=g)
    score = -torch.rand(B, W, device="cuda", generator=g).cumsum(1)
    ctx = sv.spec_beam_init(B, W, W, V, torch.bfloat16)
    token, logq, new = (torch.empty(B, W, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.float32))

    def pair(parent, state):
        sv.spec_beam_select(ctx, logits, score, None, parent, token, new, logq)
        sv.spec_beam_reorder(parent, state, state)

    parent, want = torch.zeros(B, W, dtype=torch.int32, device="cuda"), start.clone()
    pair(parent, want)
    torch.cuda.synchronize()
    assert torch.equal(want, torch.gather(start, 2, parent.long()[None, :, :, None].expand_as(start)))
    for _ in range(3):
        side = torch.cuda.Stream()
        again, state = torch.zeros_like(parent), start.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            sv.spec_beam_set_stream(ctx)
            pair(again, state)
        torch.cuda.synchronize()
        assert torch.equal(again, parent) and torch.equal(state, want)
