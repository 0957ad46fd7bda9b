"""Distillation of rows whose logits hold large finite values (spec_distill_*): rows masked with a
large constant, in part or throughout, up to the ends of the type, in either sign.

The reference takes everything against the row's largest scaled logit M: S = sum exp(x - M),
loss = sum_j p_j (log p_j - (x_j - M)) + P log S, q = exp(x - M) / S. Tolerances, as those of
ordinary rows (tests/test_gpu_distill.py) where e = 2^-23 (ln V + 6):
* lse: e, plus the rounding of M + log S to binary64 and one operation before it, 2^-52 |lse|;
* loss: P e, its rounding 2^-24 |loss|, 2^-40, and the binary64 terms of the list: each carries a
  few roundings of |x_j - M|, or (below 3e6, where the sum is not taken against M) of |x_j| and
  |M|, 2^-50 of those in all;
* gradient: |weight| r (P q (e + 2^-24 (1.5 |x - lse| + 6)) + 2^-48 p) for p the listed mass
  there, plus the roundings to binary32 and to the output's type, 2^-24 and half its epsilon;
* a value below 2^-120 may be rounded to a subnormal or to zero.
"""
import math

import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
K = 6


def make(V, dtype, full, every=1):
    """Rows: every constant, throughout, with a slightly larger one among it, with one ordinary entry
    (listed in some), and before or behind ordinary entries; at three temperatures."""
    info = torch.finfo(DTYPE[dtype])
    g = torch.Generator().manual_seed(V)
    rows, temps = [], []
    for c in (2.8e6, 3e6, 1e9, 1e10, 1e30, info.max):
        for sign in (-1.0, 1.0):
            for kind in range(5):
                z = torch.randn(V, generator=g) * 2.5
                if kind == 0:
                    z[:] = sign * c
                elif kind == 1:
                    z[:] = sign * c * (1 - 2.0 ** -7)
                    z[torch.rand(V, generator=g) < 0.3] = sign * c
                elif kind == 2:
                    z[:] = sign * c
                    z[int(torch.randint(0, V, (1,), generator=g))] = 1.5
                elif kind == 3:
                    z[:V // 2 + 1] = sign * c
                else:
                    z[V // 3:] = sign * c
                rows.append(z)
                temps.append((1.0, 2.0, 0.5)[len(rows) % 3])
    rows, temps = rows[::every], temps[::every]
    N = len(rows)
    z = torch.stack(rows).to(DTYPE[dtype])
    ids = torch.randint(0, V, (N, K), generator=g).int()
    ids[torch.rand(N, K, generator=g) < 0.2] = -1
    ids[:, 0] = z.float().abs().argmin(1).int()
    ids[::2, 0] = V - 1
    ids[::4, 1] = ids[::4, 0]
    return dict(logits=z.cuda(), ids=ids.cuda(), teacher=(torch.randn(N, K, generator=g) * 2).cuda(),
                temperature=torch.tensor(temps).cuda(), weight=torch.randn(N, generator=g).cuda(),
                teacher_lse=(torch.rand(N, generator=g).double() * 2 + 4).cuda() if full else None)


def call(d, calls, in_place):
    N, V = d["logits"].shape
    z = d["logits"].clone()
    loss, lse = torch.full((N,), 7.0, device="cuda"), torch.full((N,), 7.0, dtype=torch.float64, device="cuda")
    grad = z if in_place else torch.full_like(z, 7.0)
    a = (z, d["ids"], d["teacher"], d["teacher_lse"], d["temperature"])
    if calls == 1:
        sv.spec_distill_loss_grad(*a, d["weight"], loss, lse, grad)
    else:
        sv.spec_distill_forward(*a, loss, lse)
        sv.spec_distill_backward(*a, lse, d["weight"], grad)
    torch.cuda.synchronize()
    return loss.cpu().numpy(), lse.cpu().numpy(), grad.float().cpu().numpy()


def check(d, got):
    z, ids = d["logits"].float().cpu().numpy(), d["ids"].cpu().numpy()
    teacher, temp = d["teacher"].cpu().numpy(), d["temperature"].cpu().numpy()
    weight = d["weight"].cpu().numpy().astype(np.float64)
    half = torch.finfo(d["logits"].dtype).eps / 2
    N, V = z.shape
    e = 2.0 ** -23 * (math.log(V) + 6)
    finite = 0
    for n in range(N):
        r = np.float32(1) / temp[n]
        with np.errstate(over="ignore"):
            x = (z[n] * r).astype(np.float64)
        M = x.max()
        where = (n, z[n, 0], z[n, -1], temp[n])
        if not np.isfinite(M):
            assert np.isnan(got[0][n]) and np.isnan(got[1][n]) and np.isnan(got[2][n]).all(), where
            continue
        finite += 1
        S = np.exp(x - M).sum()
        q = np.exp(x - M) / S
        j = ids[n][ids[n] >= 0]
        y = (teacher[n] * r).astype(np.float64)[ids[n] >= 0]
        norm = y.max() + np.log(np.exp(y - y.max()).sum())
        logp = y - (norm if d["teacher_lse"] is None else d["teacher_lse"][n].item())
        p = np.exp(logp)
        P = p.sum()
        loss, lse = (p * (logp - (x[j] - M))).sum() + P * np.log(S), M + np.log(S)
        assert abs(got[1][n] - lse) <= e + 2.0 ** -52 * abs(lse), where
        tol = P * e + 2.0 ** -24 * abs(loss) + 2.0 ** -40 + 2.0 ** -50 * ((p * np.abs(x[j] - M)).sum() + P * min(abs(M), 3e6))
        if abs(loss) > 3.4e38:
            assert np.isinf(got[0][n]) or got[0][n] > 3.39e38, where
        else:
            assert abs(got[0][n] - loss) <= tol, (where, got[0][n], loss, tol)
        mass = np.zeros(V)
        np.add.at(mass, j, p)
        grad = weight[n] * r * (P * q - mass)
        away = np.minimum(np.abs(x - M - np.log(S)), 1e6)       # q is 0 long before
        near = np.abs(weight[n]) * r * (P * q * (e + 2.0 ** -24 * (1.5 * away + 6)) + 2.0 ** -48 * mass)
        tol = near + (half + 2.0 ** -24) * (np.abs(grad) + near) + 2.0 ** -120
        off = np.abs(got[2][n] - grad)
        assert (off <= tol).all(), (where, int(np.argmax(off - tol)), off.max())
    return finite


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,every", [(999, 1), (8191, 2), (20011, 1), (61001, 5), (100003, 5), (152064, 7), (300007, 11)])
def test_rows_with_large_finite_logits(V, every, dtype, full):
    print(f"\n[distill far V={V} {dtype} full={full}]", flush=True)
    d = make(V, dtype, full, every)
    for calls in (1, 2):
        got = call(d, calls, False)
        assert check(d, got) >= (5 if every < 5 else 3)
        placed = call(d, calls, True)
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, placed))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_some_of_them_far(dtype):
    """More than 256 rows (the forward pass's other shape), far rows among ordinary ones."""
    d = make(1003, dtype, False)
    N = d["logits"].shape[0]
    times = 300 // N + 1
    many = {k: None if v is None else torch.cat([v] * times) for k, v in d.items()}
    many["logits"][::7].normal_()
    for calls in (1, 2):
        check(many, call(many, calls, False))


def test_a_padded_row_of_a_large_constant_stays_zero():
    d = make(2003, "bf16", False)
    d["ids"][:] = -1
    for calls in (1, 2):
        loss, lse, grad = call(d, calls, False)
        assert (loss == 0).all() and np.isnan(lse).all() and (grad == 0).all()


def test_far_rows_replayed_from_a_graph():
    d = make(4001, "bf16", False)
    N, V = d["logits"].shape
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, dtype=torch.float64, device="cuda")
    grad = torch.empty_like(d["logits"])
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
    order = torch.randperm(N, generator=torch.Generator().manual_seed(1)).cuda()
    for _ in range(3):
        d["logits"].copy_(d["logits"][order].clone())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call(d, 2, False)
        got = (loss.cpu().numpy(), lse.cpu().numpy(), grad.float().cpu().numpy())
        assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 999, 20011, 300007])
def test_coefficients_past_the_largest_value(V, dtype):
    """weight / T (or P, of a teacher normaliser far too small) beyond binary32: entries of the gradient
    whose value is inside it have that value, masked ones are 0, the others infinite. Tolerances as
    above, with |x - lse| at most |x - M| + ln V; an exponential below 2^-120 may become zero before
    the coefficient multiplies it."""
    N = 6
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, V, generator=g)
    z[:, V - 2:] = -math.inf                              # masked
    T = torch.tensor([1e-36, 1e-36, 1.0, 1.0, 0.5, 2.0])
    z[:2] = torch.where(torch.isinf(z[:2]), z[:2], 1e-36)  # x = 1 throughout
    d = dict(logits=z.to(DTYPE[dtype]).cuda(), ids=torch.zeros(N, K, dtype=torch.int32).cuda() - 1,
             teacher=torch.zeros(N, K).cuda(), temperature=T.cuda(),
             weight=torch.tensor([1e3, -2e4, 1.0, -3.0, 3e38, -3e38]).cuda(),
             teacher_lse=torch.tensor([1.0, 1.0, -100.0, -95.0, 0.0, 0.0], dtype=torch.float64).cuda())
    d["ids"][:, 0] = 1
    largest, half = torch.finfo(DTYPE[dtype]).max, torch.finfo(DTYPE[dtype]).eps / 2
    zf, r = d["logits"].float().cpu().numpy(), np.float32(1) / T.numpy()
    e = 2.0 ** -23 * (math.log(V) + 6)
    for calls in (1, 2):
        got = call(d, calls, False)
        placed = call(d, calls, True)
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, placed))
        for n in range(N):
            x = (zf[n] * r[n]).astype(np.float64)
            M = x.max()
            q = np.exp(x - M) / np.exp(x - M).sum()
            p = math.exp(0.0 - d["teacher_lse"][n].item())
            coef = float(d["weight"][n].item()) * float(r[n])
            grad = coef * p * q
            grad[1] = coef * (p * q[1] - p)
            away = np.where(np.isinf(x), 0.0, np.abs(x - M) + math.log(V))
            near = np.abs(coef * p * q) * (e + 2.0 ** -24 * (1.5 * away + 6)) + 2.0 ** -48 * abs(coef * p) * (np.arange(V) == 1)
            inside = np.abs(grad) < 0.99 * largest
            tol = near + (half + 2.0 ** -24) * (np.abs(grad) + near) + 2.0 ** -120 * max(1.0, abs(coef * p))
            with np.errstate(invalid="ignore"):
                off = np.abs(got[2][n] - grad)
            assert (off[inside] <= tol[inside]).all(), (n, calls, int(np.argmax(np.where(inside, off - tol, -1))))
            assert (got[2][n, V - 2:] == 0).all()
            beyond = np.abs(grad) > 1.01 * largest
            assert (np.isinf(got[2][n][beyond]) & (np.sign(got[2][n][beyond]) == np.sign(grad[beyond]))).all()
