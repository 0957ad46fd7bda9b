"""GPU parity of the distillation loss and its gradient (spec_distill_*) against
oracle/draft_ops.py.

Tolerances, from the definition's arithmetic (half a step of binary32 is 2^-24):
* lse: e = 2^-23 (ln V + 6). A term 2^(x log2e - m) carries the fma's rounding (|x log2e - m|
  2^-24, in the mean over the row at most ln V log2e 2^-24, times ln 2), the exponential's last
  place 2^-23, and at most 7 * 2^-24 from a binary32 sum of 8; keeping the row in base-2 units
  of the rounded log2e moves it by at most 1.4e-8 ln V;
* loss: P e plus its rounding 2^-24, plus 2^-40 for the list's binary64 terms;
* gradient of a vocabulary entry: |weight| r P q (e + 2^-24 (1.5 |x - lse| + 6)): the row's
  normaliser, the exponent's rounding (and 1.4e-8 |x - lse| for log2e), the exponential, the
  row's coefficient and one product; plus the rounding to the output's type, half its epsilon;
* a value below 2^-120 may be rounded to a subnormal or to zero.
"""
import math

import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv
from oracle import draft_ops as ops

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(N, V, K, dtype, seed, full=False, offset=0):
    g = torch.Generator().manual_seed(seed)
    flat = torch.zeros(N * V + offset, dtype=DTYPE[dtype], device="cuda")
    flat[offset:] = (torch.randn(N * V, generator=g) * 2.5).to(DTYPE[dtype]).cuda()
    ids = torch.randint(0, V, (N, K), generator=g).int()
    ids[torch.rand(N, K, generator=g) < 0.2] = -1
    if N > 3:
        ids[1] = -1                                  # a padded row
        ids[2] = int(ids[2].max().clamp(min=0))      # one id, many times
    teacher = torch.randn(N, K, generator=g) * 2
    if K > 2:
        teacher[:, 1] = -math.inf                    # an entry without mass
    d = dict(logits=flat[offset:].view(N, V), ids=ids.cuda(), teacher=teacher.cuda(),
             temperature=(torch.rand(N, generator=g) * 1.5 + 0.5).cuda(),
             weight=torch.randn(N, generator=g).cuda(), teacher_lse=None)
    if full:
        d["teacher_lse"] = (torch.rand(N, generator=g).double() * 2 + 4).cuda()
    return d


def call(d, calls, grad=None):
    N, V = d["logits"].shape
    loss = torch.full((N,), 7.0, device="cuda")
    lse = torch.full((N,), 7.0, dtype=torch.float64, device="cuda")
    if grad is None:
        grad = torch.full((N, V), 7.0, dtype=d["logits"].dtype, device="cuda")
    a = (d["logits"], d["ids"], d["teacher"], d["teacher_lse"], d["temperature"])
    if calls == 1:
        sv.spec_distill_loss_grad(*a, d["weight"], loss, lse, grad)
    else:
        sv.spec_distill_forward(*a, loss, lse)
        sv.spec_distill_backward(*a, lse, d["weight"], grad)
    torch.cuda.synchronize()
    return loss.cpu().numpy(), lse.cpu().numpy(), grad.float().cpu().numpy()


def check(d, got, z=None):
    z = d["logits"].float().cpu().numpy() if z is None else z
    N, V = z.shape
    ids, weight = d["ids"].cpu().numpy(), d["weight"].cpu().numpy().astype(np.float64)
    temp = d["temperature"].cpu().numpy()
    tlse = None if d["teacher_lse"] is None else d["teacher_lse"].cpu().numpy()
    loss, lse, grad = ops.distill(z, ids, d["teacher"].cpu().numpy(), tlse, temp, weight)
    e = 2.0 ** -23 * (math.log(V) + 6)
    assert np.array_equal(np.isnan(got[1]), np.isnan(lse))
    live = ~np.isnan(lse)
    assert (np.abs(got[1] - lse)[live] <= e).all(), np.abs(got[1] - lse)[live].max()
    assert np.array_equal(np.isnan(got[0]), np.isnan(loss))
    assert np.array_equal(np.isinf(got[0]), np.isinf(loss))
    # the mass from the formula, for the rows that have one
    with np.errstate(all="ignore"):
        r = np.where(temp > 0, np.float32(1) / temp, 1).astype(np.float32)
        y = np.where(ids >= 0, (d["teacher"].cpu().numpy() * r[:, None]).astype(np.float64), -np.inf)
        lt = ops.row_lse(y) if tlse is None else tlse
        P = np.where(live, np.exp(y - lt[:, None]).sum(1), 0.0)
    fine = np.isfinite(loss)
    assert (np.abs(got[0] - loss)[fine] <= (P * e + 2.0 ** -24 * np.abs(loss) + 2.0 ** -40)[fine]).all()
    assert np.array_equal(np.isnan(got[2]), np.isnan(grad))
    half = torch.finfo(d["logits"].dtype).eps / 2
    for n in np.nonzero(~np.isnan(grad).any(1))[0]:
        if not live[n]:
            assert (got[2][n] == 0).all()
            continue
        x = (z[n] * r[n]).astype(np.float64)
        with np.errstate(all="ignore"):
            away = np.where(np.isneginf(x), 0.0, np.abs(x - lse[n]))
            near = np.abs(weight[n]) * r[n] * P[n] * np.exp(x - lse[n]) * (e + 2.0 ** -24 * (1.5 * away + 6))
        tol = near + half * (np.abs(grad[n]) + near) + 2.0 ** -120
        off = np.abs(got[2][n] - grad[n])
        assert (off <= tol).all(), (n, int(np.argmax(off - tol)), off.max())


SHAPES = [(1, 1, 1), (1, 2, 3), (5, 7, 4), (4, 257, 8), (6, 1000, 256), (9, 8192, 16), (5, 8193, 65),
          (3, 32000, 32), (37, 20011, 10), (4, 65536, 64), (3, 152064, 64), (2, 201088, 8), (2, 300007, 20)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", SHAPES)
def test_loss_and_gradient(N, V, K, dtype):
    print(f"\n[distill N={N} V={V} K={K} {dtype}]", flush=True)
    for full in (False, True):
        d = make(N, V, K, dtype, seed=N + V + K, full=full)
        one, two = call(d, 1), call(d, 2)
        check(d, one)
        check(d, two)


@pytest.mark.parametrize("offset,goff", [(1, 0), (3, 3), (0, 5), (7, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_alignment_of_logits_and_gradient(dtype, offset, goff):
    N, V = 5, 9001
    d = make(N, V, 12, dtype, seed=offset, offset=offset)
    for calls in (1, 2):
        buf = torch.full((N * V + goff + 16,), 7.0, dtype=DTYPE[dtype], device="cuda")
        check(d, call(d, calls, buf[goff:goff + N * V].view(N, V)))
        assert bool((buf[:goff] == 7).all()) and bool((buf[goff + N * V:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [999, 40000, 300007])
def test_gradient_in_the_logits_place(V, dtype):
    for calls in (1, 2):
        d = make(6, V, 30, dtype, seed=V)
        want = call(d, calls)
        z = d["logits"].float().cpu().numpy()
        got = call(d, calls, d["logits"])
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, want))
        check(d, got, z)


def test_sentinels_and_masks():
    for dtype in ("f32", "bf16"):
        N, V, K = 12, 5001, 6
        d = make(N, V, K, dtype, seed=3)
        d["ids"][:] = torch.arange(K).int().cuda() * 700
        z, t, ids, teacher = d["logits"], d["temperature"], d["ids"], d["teacher"]
        teacher[:] = 1.0
        t[0], t[1], t[2], t[3] = 0.0, -1.0, math.nan, math.inf
        t[4] = 1e-45                                  # its reciprocal overflows
        ids[5, 3] = V                                 # outside
        z[6] = -math.inf
        z[7, 5] = math.nan
        z[8, 6] = math.inf
        z[9, 2500:] = -math.inf                       # a masked vocabulary, two listed entries in it
        teacher[9, 4:] = -math.inf
        z[10, 700] = -math.inf                        # mass where the student has none
        teacher[11] = -math.inf                       # no mass at all
        for calls in (1, 2):
            got = call(d, calls)
            check(d, got)
            assert np.isnan(got[0][:9]).all() and np.isnan(got[2][:9]).all()
            assert np.isfinite(got[0][9]) and np.isinf(got[0][10]) and got[0][11] == 0
            assert np.isfinite(got[2][9:]).all() and (got[2][9, 2501:] == 0).all()
        d["teacher_lse"] = torch.zeros(N, dtype=torch.float64, device="cuda")
        d["teacher_lse"][9], d["teacher_lse"][10] = math.nan, -math.inf
        for calls in (1, 2):
            got = call(d, calls)
            check(d, got)
            assert np.isnan(got[0][9:11]).all()


def test_padded_rows_look_at_nothing():
    """A row without entries has loss and gradient 0 whatever its logits and temperature hold."""
    d = make(4, 1003, 5, "bf16", seed=8)
    d["ids"][0] = -1
    d["logits"][0] = math.nan
    d["temperature"][0] = math.nan
    d["teacher"][0] = math.nan
    for calls in (1, 2):
        got = call(d, calls)
        assert got[0][0] == 0 and np.isnan(got[1][0]) and (got[2][0] == 0).all()
        d2 = {k: (v[1:] if torch.is_tensor(v) else v) for k, v in d.items()}
        check(d2, tuple(x[1:] for x in got))


def test_gradient_against_central_differences_of_the_definition():
    N, V, K, h = 2, 41, 5, 1e-5
    d = make(N, V, K, "f32", seed=4)
    d["temperature"].fill_(1.0)
    got = call(d, 1)[2]
    x = d["logits"].double().cpu().numpy()
    y, ids = d["teacher"].double().cpu().numpy(), d["ids"].cpu().numpy()
    weight = d["weight"].double().cpu().numpy()
    f = lambda x: ops.distill_scaled(x, ids, y, None, weight, np.ones(N))[0]
    for v in range(V):
        step = np.zeros((N, V))
        step[:, v] = h
        slope = (f(x + step) - f(x - step)) / (2 * h) * weight
        # h^2 for the difference, 1e-9 for its rounding, 1e-6 relative to entries below 3 for binary32
        assert (np.abs(slope - got[:, v]) < h * h + 1e-9 + 3e-6).all()


def test_sum_of_the_gradient_is_zero_when_the_list_has_all_mass():
    """q and p both sum to one: the gradient's sum over the vocabulary vanishes."""
    d = make(3, 4001, 20, "f32", seed=6)
    got = call(d, 1)[2].astype(np.float64)
    e = 2.0 ** -23 * (math.log(4001) + 6)
    w = np.abs(d["weight"].cpu().numpy()) / d["temperature"].cpu().numpy()
    assert (np.abs(got.sum(1)) <= w * 4 * (e + 2.0 ** -24 * 60)).all()


def test_repeated_calls_are_equal():
    d = make(20, 30001, 40, "bf16", seed=12)
    first = call(d, 1)
    for _ in range(20):
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(first, call(d, 1)))


def test_outputs_behind_the_last_row_stay():
    N, V = 3, 1001
    d = make(N, V, 4, "bf16", seed=1)
    loss, lse = torch.full((N + 2,), 7.0, device="cuda"), torch.full((N + 2,), 7.0, dtype=torch.float64, device="cuda")
    grad = torch.full((N + 1, V), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.spec_distill_loss_grad(d["logits"], d["ids"], d["teacher"], None, d["temperature"], d["weight"],
                              loss[:N], lse[:N], grad[:N])
    torch.cuda.synchronize()
    assert (loss[N:] == 7).all() and (lse[N:] == 7).all() and (grad[N:] == 7).all()


def test_training_step_replayed_from_a_graph():
    d = make(8, 20011, 16, "bf16", seed=2)
    N, V = d["logits"].shape
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, dtype=torch.float64, device="cuda")
    grad = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    a = (d["logits"], d["ids"], d["teacher"], None, d["temperature"])

    def step():
        sv.spec_distill_forward(*a, loss, lse)
        sv.spec_distill_backward(*a, lse, d["weight"], grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(4):
        new = make(8, 20011, 16, "bf16", seed=30 + n)
        for k in ("logits", "ids", "teacher", "temperature", "weight"):
            d[k].copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call(d, 2)
        got = (loss.cpu().numpy(), lse.cpu().numpy(), grad.float().cpu().numpy())
        assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(got, want))


def test_the_heads_normaliser_serves_the_backward_call():
    """spec_lowrank_head's row normalisers (same logits and temperatures) in the place of the
    forward call's."""
    N, d_, r, V = 8, 128, 64, 4096
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    ctx = sv.spec_lowrank_head_init(N, d_, r, V)
    d = make(N, V, 9, "bf16", seed=5)
    lse = torch.empty(N, dtype=torch.float64, device="cuda")
    sv.spec_lowrank_head(ctx, bf(N, d_), bf(r, d_) * 0.1, bf(V, r) * 0.1, d["temperature"], d["logits"], lse)
    grad = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    a = (d["logits"], d["ids"], d["teacher"], None, d["temperature"])
    sv.spec_distill_backward(*a, lse, d["weight"], grad)
    loss = call(d, 1)
    live = ~np.isnan(loss[1])
    # two normalisers of one row, each within the bound above (the head's own sums are shorter)
    assert (np.abs(lse.cpu().numpy() - loss[1])[live] <= 2 * 2.0 ** -23 * (math.log(V) + 6)).all()
    check(d, (loss[0], loss[1], grad.float().cpu().numpy()))


def test_rows_past_32_bit_offsets():
    """A gradient row whose elements start more than 2^32 bytes behind the first."""
    N, V = 12, 200_000_000
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    grad = torch.full((N, V), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((N, 1), V - 1, dtype=torch.int32, device="cuda")
    f = lambda v, dt=torch.float32: torch.full((N,), v, dtype=dt, device="cuda")
    loss, lse = f(0.0), f(0.0, torch.float64)
    sv.spec_distill_loss_grad(z, ids, torch.zeros(N, 1, device="cuda"), None, f(1.0), f(1.0), loss, lse, grad)
    torch.cuda.synchronize()
    e = 2.0 ** -23 * (math.log(V) + 6)
    assert (lse - math.log(V)).abs().max().item() <= e
    assert (loss - math.log(V)).abs().max().item() <= e + 2.0 ** -24 * 20
    q = 1.0 / V
    for n in (0, N - 1):
        assert abs(grad[n, V - 1].item() - (q - 1)) <= 2.0 ** -8
        dense = grad[n, :V - 1]
        assert abs(dense.max().item() - q) <= q * 2.0 ** -7 and abs(dense.min().item() - q) <= q * 2.0 ** -7
    del z, grad, dense
    torch.cuda.empty_cache()


def test_two_calls_at_once_on_two_streams():
    ds = [make(30, 40009, 20, "bf16", seed=60 + n) for n in range(2)]
    want = [call(d, 1) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    outs = []
    torch.cuda.synchronize()
    for d, st in zip(ds, streams):
        N, V = d["logits"].shape
        o = (torch.empty(N, device="cuda"), torch.empty(N, dtype=torch.float64, device="cuda"),
             torch.empty(N, V, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        sv.spec_distill_loss_grad(d["logits"], d["ids"], d["teacher"], d["teacher_lse"], d["temperature"],
                                  d["weight"], *o, stream=st)
        outs.append(o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(np.array_equal(a.float().cpu().numpy() if a.dtype == torch.bfloat16 else a.cpu().numpy(), b,
                                  equal_nan=True) for a, b in zip(o, w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_that_rise_along_the_row(dtype):
    """The running reference is moved again and again, and far-apart logits underflow."""
    d = make(4, 70003, 12, dtype, seed=90)
    d["logits"].copy_(torch.linspace(-300, 300, 70003))
    for calls in (1, 2):
        check(d, call(d, calls))
    d["logits"].neg_()
    for calls in (1, 2):
        check(d, call(d, calls))


def test_refusals_of_the_binding():
    d = make(3, 100, 4, "f32", seed=1)
    N, V = 3, 100
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, dtype=torch.float64, device="cuda")
    f = lambda **k: sv.spec_distill_forward(*[{**d, **k}[n] for n in
                                              ("logits", "ids", "teacher", "teacher_lse", "temperature")], loss, lse)
    f()
    for bad in (dict(logits=d["logits"].double()), dict(ids=d["ids"].long()), dict(teacher=d["teacher"].bfloat16()),
                dict(teacher_lse=torch.zeros(N, device="cuda"))):
        with pytest.raises(TypeError):
            f(**bad)
    for bad in (dict(logits=d["logits"].t().contiguous().t()), dict(ids=d["ids"][:2].contiguous()),
                dict(temperature=d["temperature"].cpu()), dict(teacher=d["teacher"][:, :3].contiguous())):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(sv.SpecVerifyError):           # lists longer than the kernel takes
        f(ids=torch.zeros(N, 257, dtype=torch.int32, device="cuda"), teacher=torch.zeros(N, 257, device="cuda"))
    with pytest.raises(sv.SpecVerifyError):           # a gradient that starts inside the logits
        buf = torch.zeros((N + 1) * V, device="cuda")
        sv.spec_distill_backward(buf[:N * V].view(N, V), d["ids"], d["teacher"], None, d["temperature"], lse,
                                 d["weight"], buf[V:].view(N, V))
