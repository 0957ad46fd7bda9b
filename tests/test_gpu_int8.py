"""GPU parity of row quantisation (spec_quantize_rows) and the 8-bit product
(spec_int8_product) against oracle/draft_ops.py: the definitions name every rounding, so
8-bit values, scales and outputs are equal bit for bit."""
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


def quantize(x):
    N, D = x.shape
    q = torch.full((N, D), 99, dtype=torch.int8, device="cuda")
    s = torch.full((N,), 7.0, device="cuda")
    sv.spec_quantize_rows(x, q, s)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def check_quantize(x):
    q, s = quantize(x)
    oq, os_ = ops.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(s, os_, equal_nan=True)
    assert np.array_equal(q, oq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 5), (2, 64), (7, 100), (5, 1024), (300, 4096), (4, 4097), (2, 8192),
                                 (1, 20011), (2, 70000)])
def test_quantize(N, D, dtype):
    g = torch.Generator().manual_seed(N + D)
    x = torch.randn(N, D, generator=g) * torch.exp(torch.randn(N, 1, generator=g) * 4)
    check_quantize(x.to(DTYPE[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 3, 6])
def test_quantize_any_alignment(dtype, offset):
    g = torch.Generator().manual_seed(offset)
    buf = torch.randn(3 * 1001 + offset, generator=g).to(DTYPE[dtype]).cuda()
    x = buf[offset:].view(3, 1001)
    N, D = x.shape
    raw = torch.full((N * D + 16,), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(N, device="cuda")
    sv.spec_quantize_rows(x, raw[offset:offset + N * D].view(N, D), s)
    torch.cuda.synchronize()
    oq, os_ = ops.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(raw[offset:offset + N * D].view(N, D).cpu().numpy(), oq)
    assert np.array_equal(s.cpu().numpy(), os_)
    assert (raw[:offset] == 99).all() and (raw[offset + N * D:] == 99).all()


def test_quantize_ties_borders_and_sentinels():
    x = torch.zeros(9, 600)
    ks = torch.arange(-127, 127, dtype=torch.float32)
    x[0, 0] = 127 * 0.25
    x[0, 1:255] = (ks + 0.5) * 0.25                    # exact ties, to even
    x[1, 0] = 127 * 0.3
    s1 = np.float32(x[1, 0].item()) / np.float32(127)
    tie = ((ks.double() + 0.5) * float(s1)).float()    # as near to ties as binary32 comes
    x[1, 1:255] = tie
    x[1, 255:509] = torch.nextafter(tie, torch.tensor(math.inf))
    x[2, 5] = 1e-44                                    # the scale underflows to zero
    x[3, 5], x[3, 6] = math.inf, 1.0
    x[4, 5], x[4, 6] = math.nan, 1.0
    x[5] = -3.0
    x[6, 7] = 3e38
    x[7, :300] = torch.linspace(-1e-40, 1e-40, 300)    # subnormal values and scale
    check_quantize(x.cuda())
    check_quantize(x.to(torch.bfloat16).cuda())


def product(a, sa, w, sw, dtype, out=None):
    out = torch.full((a.shape[0], w.shape[0]), 7.0, dtype=DTYPE[dtype], device="cuda") if out is None else out
    sv.spec_int8_product(a, sa, w, sw, out)
    torch.cuda.synchronize()
    return out


def ints(shape, seed, extreme=False):
    g = torch.Generator().manual_seed(seed)
    if extreme:
        return torch.full(shape, -128, dtype=torch.int8).cuda()
    return torch.randint(-128, 128, shape, generator=g).to(torch.int8).cuda()


def check_product(a, sa, w, sw, dtype, out):
    want = torch.from_numpy(ops.int8_product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy()))
    want = want.to(DTYPE[dtype])
    assert torch.equal(out.cpu().view(torch.int32 if dtype == "f32" else torch.int16),
                       want.view(torch.int32 if dtype == "f32" else torch.int16))


SHAPES = [(1, 16, 1), (1, 64, 8), (3, 48, 5), (1, 512, 4096), (16, 1024, 1000), (17, 80, 129), (33, 256, 127),
          (64, 512, 2056), (65, 4096, 300), (128, 128, 128), (130, 144, 513), (200, 2048, 1111), (256, 512, 4099),
          (300, 4096, 520), (513, 64, 260), (1000, 192, 777)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", SHAPES)
def test_product(N, D, V, dtype):
    print(f"\n[int8 N={N} D={D} V={V} {dtype}]", flush=True)
    a, w = ints((N, D), N + D), ints((V, D), V + D + 1)
    sa, sw = torch.rand(N, device="cuda") * 0.1, torch.rand(V, device="cuda") * 0.01
    check_product(a, sa, w, sw, dtype, product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [
    (33, 48, 51203), (64, 272, 51200),           # enough columns for tiles of 128 x 64
    (65, 80, 57347), (128, 400, 57344),          # 128 x 128
    (129, 16, 28673), (300, 144, 28675), (257, 1040, 28672), (512, 2064, 30008),   # 256 x 256
])
def test_product_in_the_larger_tiles(N, D, V, dtype):
    print(f"\n[int8 N={N} D={D} V={V} {dtype}]", flush=True)
    a, w = ints((N, D), N + D), ints((V, D), V + D + 1)
    sa, sw = torch.rand(N, device="cuda") * 0.1, torch.rand(V, device="cuda") * 0.01
    check_product(a, sa, w, sw, dtype, product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("N,V", [(64, 51203), (128, 57347), (300, 28675)])
def test_the_larger_tiles_write_their_rows_only(N, V):
    D = 32
    a, w = ints((N, D), 3), ints((V, D), 4)
    sa, sw = torch.rand(N, device="cuda"), torch.rand(V, device="cuda")
    for offset in (0, 3):
        buf = torch.full((N * V + offset + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        product(a, sa, w, sw, "bf16", buf[offset:offset + N * V].view(N, V))
        check_product(a, sa, w, sw, "bf16", buf[offset:offset + N * V].view(N, V))
        assert (buf[:offset] == 7).all() and (buf[offset + N * V:] == 7).all()


@pytest.mark.parametrize("N", [1, 40, 300])
def test_product_of_the_largest_magnitudes(N):
    """Every operand -128 at the largest depth: the sums come within 2^18 of 2^31."""
    D, V = sv.SPEC_INT8_MAX_DEPTH, 40
    a, w = ints((N, D), 0, True), ints((V, D), 0, True)
    one = torch.ones(max(N, V), device="cuda")
    out = product(a, one[:N], w, one[:V], "f32")
    assert (out == float(np.float32(D * 16384))).all()


def test_product_scales_and_sentinels():
    a, w = ints((5, 64), 1), ints((70, 64), 2)
    sa, sw = torch.rand(5, device="cuda"), torch.rand(70, device="cuda")
    sa[1], sa[2], sw[3], sw[4] = 0.0, math.nan, math.inf, 0.0
    a[3] = 0
    got = product(a, sa, w, sw, "f32").cpu().numpy()
    want = ops.int8_product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[2]).all()


@pytest.mark.parametrize("offset", [1, 2, 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_product_writes_its_rows_only(dtype, offset):
    N, D, V = 35, 64, 131
    a, w = ints((N, D), 3), ints((V, D), 4)
    sa, sw = torch.rand(N, device="cuda"), torch.rand(V, device="cuda")
    buf = torch.full((N * V + offset + 64,), 7.0, dtype=DTYPE[dtype], device="cuda")
    product(a, sa, w, sw, dtype, buf[offset:offset + N * V].view(N, V))
    check_product(a, sa, w, sw, dtype, buf[offset:offset + N * V].view(N, V))
    assert (buf[:offset] == 7).all() and (buf[offset + N * V:] == 7).all()


def test_product_past_32_bit_offsets():
    """Outputs and weights more than 2^32 bytes from their start."""
    N, D, V = 24, 64, 70_000_000
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-128, 128, (V, D), device="cuda", generator=g, dtype=torch.int8)
    a = ints((N, D), 5)
    sa, sw = torch.rand(N, device="cuda"), torch.rand(V, device="cuda", generator=g)
    out = product(a, sa, w, sw, "f32")
    for v in (0, 1 << 24, V - 300):
        check_product(a, sa, w[v:v + 300].contiguous(), sw[v:v + 300].contiguous(), "f32", out[:, v:v + 300].contiguous())
    del out, w
    torch.cuda.empty_cache()


def test_quantised_product_is_near_the_real_one():
    """Both operands quantised: each product term is off by at most half a step of either side,
    |x| sw / 2 + |w| sa / 2 + sa sw / 4 for values within 127 steps."""
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(20, 512, generator=g).cuda(), torch.randn(300, 512, generator=g).cuda()
    qx, qw = torch.empty(20, 512, dtype=torch.int8, device="cuda"), torch.empty(300, 512, dtype=torch.int8, device="cuda")
    sx, sw = torch.empty(20, device="cuda"), torch.empty(300, device="cuda")
    sv.spec_quantize_rows(x, qx, sx)
    sv.spec_quantize_rows(w, qw, sw)
    got = product(qx, sx, qw, sw, "f32").double().cpu()
    xd, wd = x.double().cpu(), w.double().cpu()
    want = xd @ wd.t().contiguous()
    sx, sw = sx.double().cpu()[:, None], sw.double().cpu()[None, :]
    bound = (xd.abs().sum(1)[:, None] * sw + wd.abs().sum(1)[None, :] * sx) / 2 + 512 * sx * sw / 4
    assert ((got - want).abs() <= bound * (1 + 1e-5) + 1e-4 * want.abs().max() * 2.0 ** -10).all()


def test_quantise_and_product_replayed_from_a_graph():
    N, D, V = 33, 256, 1003
    x = torch.randn(N, D, device="cuda").to(torch.bfloat16)
    w, sw = ints((V, D), 7), torch.rand(V, device="cuda")
    q, s = torch.empty(N, D, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    out = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")

    def step():
        sv.spec_quantize_rows(x, q, s)
        sv.spec_int8_product(q, s, w, sw, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(4):
        x.copy_(torch.randn(N, D, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        oq, os_ = ops.quantize_rows(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_)
        check_product(q, s, w, sw, "bf16", out)
        eager = torch.empty_like(out)
        sv.spec_int8_product(q, s, w, sw, eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def test_refusals_of_the_binding():
    a, w = ints((4, 32), 1), ints((6, 32), 2)
    sa, sw, out = torch.rand(4, device="cuda"), torch.rand(6, device="cuda"), torch.empty(4, 6, device="cuda")
    for bad in ((a.int(), sa, w, sw, out), (a, sa.double(), w, sw, out), (a, sa, w, sw, out.half())):
        with pytest.raises(TypeError):
            sv.spec_int8_product(*bad)
    for bad in ((a, sa, w[:, :16].contiguous(), sw, out), (a, sa, w, sw[:3], out), (a, sa, w, sw, out.t()),
                (a, sa, w, sw, torch.empty(6, 4, device="cuda").t()), (a.cpu(), sa, w, sw, out)):
        with pytest.raises(ValueError):
            sv.spec_int8_product(*bad)
    with pytest.raises(sv.SpecVerifyError):            # a depth that is no multiple of 16
        sv.spec_int8_product(ints((4, 24), 1), sa, ints((6, 24), 2), sw, out)
    with pytest.raises(sv.SpecVerifyError):            # rows that are not 16-byte aligned
        buf = torch.zeros(4 * 32 + 4, dtype=torch.int8, device="cuda")
        sv.spec_int8_product(buf[4:].view(4, 32), sa, w, sw, out)
