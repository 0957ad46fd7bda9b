"""GPU parity of the token scores (spec_token_logprobs) and their gradient
(spec_token_logprobs_backward) against oracle/draft_ops.py.

Ranks, tokens and the largest scaled logit are equal. Bounds, with u = 2^-24 (half a step of
binary32), d = x - M, p the probabilities:
* an exponential is off by at most e_v = 2^-22 (1 + |d_v|) of itself: |d| times half a step for
  each of d, the constant and the product (3 u |d|), a step of the exponential;
* log S: D = 2^-23 (ln V + 6), which the header states, and u |log S| when it is handed out;
* logprob: D and u |logprob|;
* entropy log S - T / S, T = sum e d: its derivative for e_v is p_v (1 - d_v + T / S) / e_v; the
  products and sums of a load add 4 u |T / S|: E = sum p e_v (1 + |d| + |T / S|) + 4 u |T / S|, and
  u of the result;
* gradient: with l = log p, c = |a| + |b| (|l| + H): p carries P = D + u log S + 2^-22 (1 + |l|), l
  the same but for its exponential, H carries E + u H; the three products and sums 3 u: r p (c (P +
  3 u) + |b| (P + E + u H)), and half a step of the type."""
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
NAMES = ("logprob", "rank", "entropy", "top_token", "top_logprob", "norm")


def outputs(N, K, dev="cuda"):
    f = lambda *s: torch.full(s, 7.0, device=dev)
    i = lambda *s: torch.full(s, 77, dtype=torch.int32, device=dev)
    return [f(N), i(N), f(N), i(N, K) if K else None, f(N, K) if K else None, f(N, 2)]


def scores(z, token, temperature, K, ctx=None):
    """z, token, temperature on the device; a dict of numpy arrays."""
    N, V = z.shape
    ctx = ctx or sv.spec_logprobs_init(N, V, K, z.dtype)
    out = outputs(N, K)
    sv.spec_token_logprobs(ctx, z, token, temperature, *out)
    torch.cuda.synchronize()
    return {k: None if t is None else t.cpu().numpy() for k, t in zip(NAMES, out)}


def bounds(z, temperature):
    """D [1], E [N], and p, l, H of rows with a finite largest entry, float64."""
    x, _ = ops.score_scaled(z, temperature)
    with np.errstate(all="ignore"):
        m = x.max(1)
        ok = np.isfinite(m) & ~np.isnan(x).any(1)
        x = np.where(ok[:, None], x, np.float32(0))
        d = x.astype(np.float64) - x.max(1).astype(np.float64)[:, None]
        l, p, h = ops.score_parts(x)
        ad = np.where(p > 0, np.abs(d), 0.0)
        mean = (p * ad).sum(1)
        D = 2.0 ** -23 * (np.log(z.shape[1]) + 6)
        E = (p * 2.0 ** -22 * (1 + ad) * (1 + ad + mean[:, None])).sum(1) + 4 * U * mean
    return ok, D, E, p, l, h


def near(got, want, off, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    assert np.isfinite(got[fine]).all(), what
    off = np.broadcast_to(off, want.shape)[fine] + U * np.abs(want[fine])
    bad = np.abs(got[fine] - want[fine]) > off
    assert not bad.any(), (what, got[fine][bad][:5], want[fine][bad][:5], off[bad][:5])


def check(z, token, temperature, K, got):
    zf = z.float().cpu().numpy()
    token, temperature = token.cpu().numpy(), None if temperature is None else temperature.cpu().numpy()
    want = ops.token_scores(zf, token, temperature, K)
    _, D, E, *_ = bounds(zf, temperature)
    assert np.array_equal(got["rank"], want["rank"])
    near(got["logprob"], want["logprob"], D, "logprob")
    near(got["entropy"], want["entropy"], E, "entropy")
    near(got["norm"][:, 0], want["norm"][:, 0], 0, "largest")
    near(got["norm"][:, 1], want["norm"][:, 1], D, "log sum")
    if K:
        assert np.array_equal(got["top_token"], want["top_token"])
        near(got["top_logprob"], want["top_logprob"], D, "top")


def rows(N, V, seed, spread=2.5, masked=0.25):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * spread
    some = torch.rand(N, 1, generator=g) < masked
    z[some & (torch.rand(N, V, generator=g) < torch.rand(N, 1, generator=g))] = -float("inf")
    token = torch.randint(0, V, (N,), generator=g).to(torch.int32)
    best = z.argmax(1).to(torch.int32)
    token = torch.where(torch.rand(N, generator=g) < 0.3, best, token)
    token[torch.rand(N, generator=g) < 0.1] = -1
    temperature = torch.where(torch.rand(N, generator=g) < 0.4, 1.0, torch.rand(N, generator=g) * 1.5 + 0.5)
    return z, token.cuda(), temperature.cuda()


SIZES = [(1, 1, 1), (3, 2, 4), (2, 7, 64), (5, 63, 1), (4, 1000, 20), (3, 8191, 64), (2, 8200, 17), (37, 20011, 5),
         (1, 32000, 50), (9, 33000, 49), (2, 128256, 20), (3, 201088, 64), (130, 5000, 16), (1, 16384, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", SIZES)
def test_scores(N, V, K, dtype):
    print(f"\n[scores N={N} V={V} K={K} {dtype}]", flush=True)
    z, token, temperature = rows(N, V, N + V + K)
    z = z.to(DTYPE[dtype]).cuda()
    check(z, token, temperature, K, scores(z, token, temperature, K))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", [(1024, 2500, 64), (1500, 9000, 8), (1030, 33000, 20), (600, 20000, 3),
                                   (640, 20011, 64), (641, 20011, 64), (256, 60000, 33)])
def test_scores_of_many_rows(N, V, K, dtype):
    print(f"\n[scores N={N} V={V} K={K} {dtype}]", flush=True)
    z, token, temperature = rows(N, V, N + V + K)
    z = z.to(DTYPE[dtype]).cuda()
    got = scores(z, token, temperature, K)
    at = np.unique(np.concatenate((np.arange(0, N, 13), np.nonzero(got["rank"] < 0)[0][:20], [N - 1])))
    sub = torch.from_numpy(at).cuda()
    check(z[sub], token[sub], temperature[sub], K, {k: v[at] for k, v in got.items()})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [2, 1100])
def test_scores_without_lists_or_temperatures(N, dtype):
    z, token, _ = rows(N, 9001, 5)
    z = z.to(DTYPE[dtype]).cuda()
    got = scores(z, token, None, 0)
    at = np.arange(0, N, 7)
    sub = torch.from_numpy(at).cuda()
    check(z[sub], token[sub], None, 0, {k: None if v is None else v[at] for k, v in got.items()})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 3, 6])
def test_any_alignment(dtype, offset):
    z, token, temperature = rows(5, 9001, offset)
    buf = torch.full((5 * 9001 + 16,), 50.0, dtype=DTYPE[dtype], device="cuda")   # what lies around is larger
    at = buf[offset:offset + 5 * 9001].view(5, 9001)
    at.copy_(z)
    check(at, token, temperature, 20, scores(at, token, temperature, 20))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [2, 1030])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two levels", "zeros", "denormals", "late", "sparse"])
def test_orders_that_crowd_the_lists(kind, N, dtype):
    V, K = 18001, 64
    v = torch.arange(V, dtype=torch.float32)
    z = dict(equal=torch.full((V,), 3.0), rising=v / 1000, falling=-v / 1000,
             zeros=torch.where(v % 3 == 1, -0.0, 0.0), late=torch.where(v >= V - 700, 5.0, -5.0) + v / 40000,
             sparse=torch.where(v % 997 == 0, v / V, -float("inf")))
    z["denormals"] = torch.tensor([-1e-45, -0.0, 0.0, 1e-45, -3e-45])[(v % 5).long()]   # -0 and +0 are one logit
    z["two levels"] = torch.where(v % 5 == 2, 1.0, 0.0)
    z = z[kind].repeat(N, 1).to(DTYPE[dtype]).cuda()
    token = (torch.arange(N, device="cuda", dtype=torch.int32) * 7919) % V
    got = scores(z, token, None, K)
    at = np.arange(0, N, 103)
    sub = torch.from_numpy(at).cuda()
    check(z[sub], token[sub], None, K, {k: v[at] for k, v in got.items()})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_tokens_at_the_ends_of_rows(dtype):
    """Their rank counts what is masked in front of them too, once."""
    for V in (9001, 9003, 9006, 20005):
        z = torch.randn(40, V, generator=torch.Generator().manual_seed(V)).to(DTYPE[dtype])
        token = torch.cat((torch.arange(20), torch.arange(V - 20, V))).int().cuda()
        z[:, :25] = z[:, V - 25:] = -float("inf")
        z = z.cuda()
        check(z, token, None, 4, scores(z, token, None, 4))


def test_lists_longer_than_what_is_there():
    z = torch.full((3, 20000), -float("inf"))
    z[0, 5000:5003] = torch.tensor([1.0, 3.0, 2.0])
    z[1, 19999] = 0.0
    z[2, :] = -1.0
    z = z.cuda()
    token = torch.tensor([5001, 0, 19999], dtype=torch.int32, device="cuda")
    got = scores(z, token, None, 64)
    check(z, token, None, 64, got)
    assert got["top_token"][0, :4].tolist() == [5001, 5002, 5000, -1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [11, 20003])
def test_empty_and_bad_rows(V, dtype):
    N = 14
    z, _, temperature = rows(N, V, 9, masked=0.0)
    token = torch.full((N,), 1, dtype=torch.int32)
    inf, nan = float("inf"), float("nan")
    z[0], z[1] = -inf, -inf
    token[1] = -1
    z[2, V // 2], z[3, V // 2], z[4, 1] = nan, inf, nan
    z[5, 0] = -nan
    z[6, 1] = -inf                                    # the token itself is masked
    z[7] = -inf
    z[7, 0] = -nan
    token[8], token[9] = V, -7
    temperature = temperature.cpu()
    for n, t in ((10, 0.0), (11, -1.0), (12, nan), (13, 1e-45)):
        temperature[n] = t
    z = z.to(DTYPE[dtype]).cuda()
    bits = z[5, 0].clone()
    z[7, 0], z[5, 0] = -bits.abs(), -bits.abs()       # a NaN with its sign set
    token, temperature = token.cuda(), temperature.cuda()
    got = scores(z, token, temperature, 5)
    check(z, token, temperature, 5, got)
    assert got["rank"].tolist()[:6] == [-1] * 6 and got["logprob"][0] == -inf and got["logprob"][1] == 0
    a = torch.ones(N, device="cuda")
    g = gradient(z, token, temperature, got, a, a)
    check_gradient(z, token, temperature, a, a, g, got)
    assert (g[:2] == 0).all() and torch.isnan(g[2:6]).all() and torch.isnan(g[10:]).all()


def gradient(z, token, temperature, got, a, b, out=None):
    N, V = z.shape
    ctx = sv.spec_logprobs_init(N, V, 0, z.dtype)
    out = torch.full_like(z, 7.0) if out is None else out
    sv.spec_token_logprobs_backward(ctx, z, token, temperature, torch.from_numpy(got["norm"]).cuda(),
                                    torch.from_numpy(got["entropy"]).cuda(), a, b, out)
    torch.cuda.synchronize()
    return out


def check_gradient(z, token, temperature, a, b, out, got):
    zf, dtype = z.float().cpu().numpy(), z.dtype
    token = token.cpu().numpy()
    temperature = None if temperature is None else temperature.cpu().numpy()
    a = a.cpu().numpy()
    b = np.zeros_like(a) if b is None else b.cpu().numpy()
    want = ops.token_scores_grad(zf, token, temperature, a, b)
    ok, D, E, p, l, h = bounds(zf, temperature)
    _, r = ops.score_scaled(zf, temperature)
    _, log_s = ops.row_parts(np.where(ok[:, None], ops.score_scaled(zf, temperature)[0], 0))
    al = np.where(p > 0, np.abs(l), 0.0)
    P = D + U * np.abs(log_s)[:, None] + 2.0 ** -22 * (1 + al)
    aa, ab = np.abs(np.where(token >= 0, a, 0.0))[:, None], np.abs(b)[:, None]
    c = aa + ab * (al + h[:, None])
    off = p * (c * (P + 3 * U) + ab * (P + E[:, None] + U * h[:, None])) * np.where(ok, r, 0)[:, None]
    g = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    half = U if dtype == torch.float32 else 2.0 ** -8
    tiny = 2.0 ** -133                                # below it both types have run out of steps
    with np.errstate(invalid="ignore"):
        bad = np.abs(g - want) > off + half * (np.abs(want) + off) + tiny
    assert not bad.any(), (g[bad][:5], want[bad][:5], np.argwhere(bad)[:5])


@pytest.mark.parametrize("bonus", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (5, 63), (4, 1000), (3, 8191), (37, 20011), (2, 128256), (1100, 300)])
def test_gradient(N, V, dtype, bonus):
    print(f"\n[gradient N={N} V={V} {dtype}]", flush=True)
    z, token, temperature = rows(N, V, N + V)
    z = z.to(DTYPE[dtype]).cuda()
    a = torch.randn(N, device="cuda")
    b = torch.randn(N, device="cuda") if bonus else None
    t = temperature if bonus else None
    got = scores(z, token, t, 0)
    out = gradient(z, token, t, got, a, b)
    check_gradient(z, token, t, a, b, out, got)
    # in the logits' place
    same = z.clone()
    gradient(same, token, t, got, a, b, same)
    assert torch.equal(same.view(torch.int16 if dtype == "bf16" else torch.int32),
                       out.view(torch.int16 if dtype == "bf16" else torch.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("x_offset,g_offset", [(1, 1), (3, 0), (0, 5)])
def test_gradient_any_alignment_and_its_rows_only(dtype, x_offset, g_offset):
    N, V = 5, 9001
    z, token, temperature = rows(N, V, 1)
    buf = torch.full((N * V + 16,), 50.0, dtype=DTYPE[dtype], device="cuda")
    x = buf[x_offset:x_offset + N * V].view(N, V)
    x.copy_(z)
    raw = torch.full((N * V + 64,), 7.0, dtype=DTYPE[dtype], device="cuda")
    a, b = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    got = scores(x, token, temperature, 0)
    out = gradient(x, token, temperature, got, a, b, raw[g_offset:g_offset + N * V].view(N, V))
    check_gradient(x, token, temperature, a, b, out, got)
    assert (raw[:g_offset] == 7).all() and (raw[g_offset + N * V:] == 7).all()


@pytest.mark.parametrize("far", [5e3, 1e7, -1e9, 1e30, -3e38])
def test_far_rows(far):
    """Rows that a mask of a large finite constant shifts or covers: the sum and the largest entry stay apart."""
    V = 9001
    z = torch.zeros(4, V)
    z[0] = far
    z[1] = far
    z[1, 17] = float(np.nextafter(np.float32(far), np.float32(np.inf)))
    z[2] = float(np.finfo(np.float32).min)                              # binary32's lowest value everywhere
    z[3] = float(np.finfo(np.float32).min)
    z[3, 5:8] = torch.tensor([1.0, 2.0, 3.0])
    token = torch.tensor([4, 17, 9, 6], dtype=torch.int32, device="cuda")
    for dtype in ("f32", "bf16"):
        x = z.to(DTYPE[dtype]).cuda()                 # of bf16 the lowest value becomes -inf
        got = scores(x, token, None, 4)
        check(x, token, None, 4, got)
        a, b = torch.tensor([1.0, -2.0, 0.5, 3.0], device="cuda"), torch.tensor([0.3, 0.0, -1.0, 2.0], device="cuda")
        check_gradient(x, token, None, a, b, gradient(x, token, None, got, a, b), got)


@pytest.mark.parametrize("T", [1e-30, 1e-3, 1e3, 3e38])
def test_extreme_temperatures(T):
    z, token, _ = rows(6, 3001, 3)
    z = z.cuda()
    temperature = torch.full((6,), T, device="cuda")
    got = scores(z, token, temperature, 8)
    check(z, token, temperature, 8, got)
    a = torch.randn(6, device="cuda") * 1e-8
    if T > 1e-20:
        check_gradient(z, token, temperature, a, a, gradient(z, token, temperature, got, a, a), got)


def test_extreme_weights():
    """Weights whose products pass binary32 where the gradient itself does not."""
    z, token, _ = rows(6, 3001, 3, masked=1.0)
    z = z.cuda()
    a = torch.tensor([3e38, 1e36, 0.0, 1e-38, -3e38, 1e31], device="cuda")
    b = torch.tensor([0.0, 1e36, 1e37, 1e-38, 1e30, -1e35], device="cuda")
    got = scores(z, token, None, 0)
    check_gradient(z, token, None, a, b, gradient(z, token, None, got, a, b), got)


def test_gradient_against_differences():
    """Central differences of the scores themselves along random directions of +-1: with |z| <= 2
    and 50 entries |l| <= 2 + 2 + ln 50 < 8, the third derivatives of logprob and entropy along the
    direction are below 16 and 200 (cumulants up to the third and fourth order of a variable within
    2 of its mean, those of the entropy times |l|), so the remainder is below h^2 / 6 of that; the
    differences' own rounding is (D + E + 2 u 8) / h."""
    N, V, h = 8, 50, 2.0 ** -6
    g = torch.Generator().manual_seed(1)
    z = ((torch.rand(N, V, generator=g) * 4 - 2) * 1024).round() / 1024
    token = torch.randint(0, V, (N,), generator=g).to(torch.int32).cuda()
    zf = z.numpy()
    _, D, E, *_ = bounds(zf, None)
    got = scores(z.cuda(), token, None, 0)
    one, none = torch.ones(N, device="cuda"), torch.zeros(N, device="cuda")
    grads = [gradient(z.cuda(), token, None, got, a, b).double().cpu() for a, b in ((one, None), (none, one))]
    for k in range(4):
        way = torch.where(torch.rand(N, V, generator=g) < 0.5, -1.0, 1.0)
        up, down = (scores((z + s * h * way).cuda(), token, None, 0) for s in (1, -1))
        for name, grad, third in (("logprob", grads[0], 16), ("entropy", grads[1], 200)):
            slope = (up[name].astype(np.float64) - down[name].astype(np.float64)) / (2 * h)
            want = (grad * way.double()).sum(1).numpy()
            assert (np.abs(slope - want) <= h * h / 6 * third + (D + E + 16 * U) / h + 1e-5).all()


def test_fewer_rows_than_the_context_has():
    ctx = sv.spec_logprobs_init(2000, 9001, 20, torch.bfloat16)
    for N in (2000, 1, 700, 1024, 3, 1023):
        z, token, temperature = rows(N, 9001, N)
        z = z.bfloat16().cuda()
        got = scores(z, token, temperature, 20, ctx)
        at = np.arange(0, N, max(1, N // 20))
        sub = torch.from_numpy(at).cuda()
        check(z[sub], token[sub], temperature[sub], 20, {k: v[at] for k, v in got.items()})


def test_the_same_bits_on_every_call():
    for N, V, K in ((3, 128256, 20), (1100, 20011, 64)):
        z, token, temperature = rows(N, V, 4)
        z = z.bfloat16().cuda()
        ctx = sv.spec_logprobs_init(N, V, K, z.dtype)
        first = scores(z, token, temperature, K, ctx)
        for _ in range(3):
            again = scores(z, token, temperature, K, ctx)
            for k in NAMES:
                assert np.array_equal(first[k], again[k], equal_nan=True)


def test_replayed_from_a_graph():
    N, V, K = 5, 33000, 20
    z, token, temperature = rows(N, V, 6)
    z = z.bfloat16().cuda()
    side = torch.cuda.Stream()
    ctx = sv.spec_logprobs_init(N, V, K, z.dtype, stream=side)
    out, grad = outputs(N, K), torch.empty_like(z)
    a = torch.randn(N, device="cuda")

    def step():
        sv.spec_token_logprobs(ctx, z, token, temperature, *out)
        sv.spec_token_logprobs_backward(ctx, z, token, temperature, out[5], out[2], a, a, grad)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        new, t, _ = rows(N, V, 60 + i)
        z.copy_(new)
        token.copy_(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: x.cpu().numpy() for k, x in zip(NAMES, out)}
        check(z, token, temperature, K, got)
        check_gradient(z, token, temperature, a, a, grad, got)
        eager = scores(z, token, temperature, K)
        for k in NAMES:
            assert np.array_equal(eager[k], got[k], equal_nan=True)


def test_two_contexts_on_two_streams():
    N, V, K = 4, 40000, 30
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = []
    for i in range(2):
        z, token, temperature = rows(N, V, 20 + i)
        inputs.append((z.bfloat16().cuda(), token, temperature))
    torch.cuda.synchronize()
    ctxs = [sv.spec_logprobs_init(N, V, K, torch.bfloat16, stream=s) for s in streams]
    outs = [outputs(N, K) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            sv.spec_token_logprobs(ctxs[i], *inputs[i], *outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(*inputs[i], K, {k: x.cpu().numpy() for k, x in zip(NAMES, outs[i])})


def test_rows_past_32_bit_offsets():
    N, V = 12000, 201088                              # 4.8 GB of logits
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for n in range(0, N, 2000):
        z[n:n + 2000] = torch.randn(2000, V, device="cuda", generator=g)
    token = torch.randint(0, V, (N,), device="cuda", generator=g).to(torch.int32)
    got = scores(z, token, None, 4)
    a = torch.randn(N, device="cuda", generator=g)
    out = gradient(z, token, None, got, a, a)
    for n in (0, 5339, 10678, N - 2):
        sub = {k: v[n:n + 2] for k, v in got.items()}
        check(z[n:n + 2], token[n:n + 2], None, 4, sub)
        check_gradient(z[n:n + 2], token[n:n + 2], None, a[n:n + 2], a[n:n + 2], out[n:n + 2], sub)
    del z, out
    torch.cuda.empty_cache()


def test_no_rows():
    ctx = sv.spec_logprobs_init(4, 100, 3, torch.float32)
    z = torch.empty(0, 100, device="cuda")
    token, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    out = outputs(0, 3)
    sv.spec_token_logprobs(ctx, z, token, None, *out)
    sv.spec_token_logprobs_backward(ctx, z, token, None, out[5], out[2], f, None, z)


def test_refusals_of_the_binding():
    N, V, K = 4, 100, 3
    ctx = sv.spec_logprobs_init(N, V, K, torch.float32)
    z, token, temperature = rows(N, V, 1)
    z = z.cuda()
    out = outputs(N, K)

    def call(**new):
        args = dict(z=z, token=token, t=temperature, **dict(zip(NAMES, out)))
        args.update(new)
        sv.spec_token_logprobs(ctx, *args.values())

    call()
    for name, bad in (("z", z.bfloat16()), ("token", token.long()), ("t", temperature.double()), ("rank", out[0]),
                      ("norm", out[5].double()), ("top_token", out[4])):
        with pytest.raises(TypeError):
            call(**{name: bad})
    for name, bad in (("z", z[:, :99].contiguous()), ("z", torch.zeros(5, V, device="cuda")), ("z", z.cpu()),
                      ("token", token[:3]), ("norm", torch.empty(2, N, device="cuda")), ("top_token", None),
                      ("z", torch.zeros(V, N, device="cuda").t())):
        with pytest.raises(ValueError):
            call(**{name: bad})
    with pytest.raises(sv.SpecVerifyError):
        call(entropy=None)
    a = torch.ones(N, device="cuda")
    with pytest.raises(sv.SpecVerifyError):            # a gradient that overlaps the logits, but is not them
        buf = torch.zeros(N * V + 8, device="cuda")
        sv.spec_token_logprobs_backward(ctx, buf[:N * V].view(N, V), token, None, out[5], out[2], a, None,
                                        buf[8:].view(N, V))
    with pytest.raises(ValueError):
        sv.spec_token_logprobs_backward(ctx, z, token, None, out[5], out[2], a[:2], None, z)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_logprobs_init(4, 100, 65, torch.float32)
    torch.cuda.synchronize()
