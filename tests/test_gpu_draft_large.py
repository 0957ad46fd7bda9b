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


def test_quantisation_of_so_many_rows_that_wide_workgroups_do_not_fit():
    """2^22 rows that 1024 threads would each take: one dispatch does not hold 2^32 work-items."""
    N, D, step = 1 << 22, 8200, 1 << 16
    print("\n[quantise 2^22 rows]", flush=True)
    x = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for n in range(0, N, step):
        x[n:n + step].normal_(0, 1 + n / N, generator=g)
    q = torch.full((N, D), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((N,), 7.0, device="cuda")
    sv.spec_quantize_rows(x, q, scale)
    torch.cuda.synchronize()
    wrong_scales, wrong_bytes = torch.zeros(2, dtype=torch.int64, device="cuda")
    for n in range(0, N, step):
        part, s = x[n:n + step], scale[n:n + step]
        # in binary64, rounded once: torch divides by a number through its reciprocal
        wrong_scales += (s != (part.abs().amax(1).double() / 127).float()).sum()
        # the bytes of the first and last 2^12 rows of each 2^16
        for a in (0, step - 4096):
            rows = slice(a, a + 4096)
            want = (part[rows].double() / s[rows].double()[:, None]).round().clamp(-127, 127)
            wrong_bytes += (want != q[n:n + step][rows]).sum()
    assert wrong_scales.item() == 0 and wrong_bytes.item() == 0


def test_distillation_in_two_calls_past_32_bit_offsets():
    """Rows whose elements start more than 2^32 bytes behind the first, through the forward pass and
    the backward pass with its rows and parts of rows."""
    N, V = 12, 200_000_000
    print("\n[distill two calls, 12 x 2e8]", flush=True)
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    z[:, V // 2:] = 1.0
    grad = torch.full((N, V), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((N, 1), V - 1, dtype=torch.int32, device="cuda")
    f = lambda v, dt=torch.float32: torch.full((N,), v, dtype=dt, device="cuda")
    loss, lse = f(0.0), f(0.0, torch.float64)
    a = (z, ids, torch.zeros(N, 1, device="cuda"), None, f(1.0))
    sv.spec_distill_forward(*a, loss, lse)
    sv.spec_distill_backward(*a, lse, f(1.0), grad)
    torch.cuda.synchronize()
    e = 2.0 ** -23 * (math.log(V) + 6)
    want = math.log(V // 2 * (1 + math.e))
    assert (lse - want).abs().max().item() <= e
    assert (loss - (want - 1)).abs().max().item() <= e + 2.0 ** -24 * 20
    for n in range(N):
        assert abs(grad[n, V - 1].item() - (math.exp(1 - want) - 1)) <= 2.0 ** -8
        for part, q in ((grad[n, :V // 2], math.exp(-want)), (grad[n, V // 2:V - 1], math.exp(1 - want))):
            assert abs(part.max().item() - q) <= q * 2.0 ** -7 and abs(part.min().item() - q) <= q * 2.0 ** -7


def test_reordering_into_another_array_past_32_bit_offsets():
    """States that start more than 2^32 bytes behind the first, in both arrays."""
    L, B, W, K, S = 3, 2, 4, 5, 1 << 28
    print("\n[reorder 3 x 2 x (4 -> 5) states of 256 MiB]", flush=True)
    src = torch.empty(L, B, W, S // 4, dtype=torch.int32, device="cuda")
    for i, state in enumerate(src.view(L * B * W, S // 4)):
        state.copy_(torch.arange(S // 4, dtype=torch.int32, device="cuda")).mul_(i + 1)
    dst = torch.full((L, B, K, S // 4), -1, dtype=torch.int32, device="cuda")
    parent = torch.tensor([[3, 0, 0, -1, 2], [1, 3, 7, 2, 1]], dtype=torch.int32, device="cuda")
    sv.spec_beam_reorder(parent, src, dst)
    torch.cuda.synchronize()
    for l in range(L):
        for b in range(B):
            for j, w in enumerate(parent[b].tolist()):
                if 0 <= w < W:
                    assert torch.equal(dst[l, b, j], src[l, b, w]), (l, b, j)
                else:
                    assert (dst[l, b, j] == -1).all(), (l, b, j)
