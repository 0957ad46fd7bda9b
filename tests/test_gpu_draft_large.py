"""The draft side's operators at sizes whose offsets pass 32 bits: the longest rows, and many rows."""
import math

import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _free_memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("calls", [1, 2])
def test_distillation_of_the_longest_row(calls):
    """2^31 - 1 entries that start off a 16-byte boundary, with the row's last and first entries listed:
    an entry's place counted from the boundary passes 2^31."""
    V, off = (1 << 31) - 1, 5
    print(f"\n[distill longest row, calls={calls}]", flush=True)
    z = torch.zeros(V + off + 3, dtype=torch.bfloat16, device="cuda")
    grad = torch.full((V + off + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    row, out = z[off:off + V].view(1, V), grad[off:off + V].view(1, V)
    ids = torch.tensor([[V - 1, 0, V - 2, V - 9]], dtype=torch.int32, device="cuda")
    f = lambda v, dt=torch.float32: torch.full((1,), v, dtype=dt, device="cuda")
    loss, lse = f(7.0), f(7.0, torch.float64)
    a = (row, ids, torch.zeros(1, 4, device="cuda"), None, f(1.0))
    if calls == 1:
        sv.spec_distill_loss_grad(*a, f(1.0), loss, lse, out)
    else:
        sv.spec_distill_forward(*a, loss, lse)
        sv.spec_distill_backward(*a, lse, f(1.0), out)
    torch.cuda.synchronize()
    e = 2.0 ** -23 * (math.log(V) + 6)
    assert abs(lse.item() - math.log(V)) <= e
    want = math.log(0.25) + math.log(V)               # four entries of 1/4 each
    assert abs(loss.item() - want) <= e + 2.0 ** -24 * want + 2.0 ** -40
    q = 1.0 / V
    for v in ids[0].tolist():
        assert abs(out[0, v].item() - (q - 0.25)) <= 2.0 ** -8 * 0.25
        out[0, v] = q
    for part in out[0].split(1 << 29):
        assert abs(part.max().item() - q) <= q * 2.0 ** -7 and abs(part.min().item() - q) <= q * 2.0 ** -7
    assert (grad[:off] == 7).all() and (grad[off + V:] == 7).all()
