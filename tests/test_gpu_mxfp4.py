"""GPU parity of the 4-bit quantisation (spec_mxfp4_quantize_rows) and product
(spec_mxfp4_product) against oracle/draft_ops.py. Codes, scales and values are exact by
definition, hence equal. The product's sum is within D' / 64 * 2^-23 of sum |a w| (the header's
bound), and rounded once more to the output's type."""
import numpy as np
import pytest
import torch

import device_draft_verification_amd as sv
from oracle import draft_ops as ops

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def quantize(x, values=True):
    N, D = x.shape
    whole = sv.spec_mxfp4_padded(D)
    q = torch.full((N, whole // 2), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((N, whole // 32), 99, dtype=torch.uint8, device="cuda")
    v = torch.full((N, D), 7.0, dtype=x.dtype, device="cuda") if values else None
    sv.spec_mxfp4_quantize_rows(x, q, s, v)
    torch.cuda.synchronize()
    return q, s, v


def check_quantize(x):
    oq, os_, ov = ops.mxfp4_quantize(x.float().cpu().numpy())
    for values in (False, True):
        q, s, v = quantize(x, values)
        assert np.array_equal(s.cpu().numpy(), os_)
        assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(v.double().cpu().numpy(), ov, equal_nan=True)


SIZES = [(1, 1), (3, 5), (2, 32), (2, 33), (5, 95), (7, 100), (4, 128), (3, 129), (5, 1024), (300, 4096), (4, 4097),
         (2, 8192), (1, 20011), (1000, 8), (2, 70000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", SIZES)
def test_quantize(N, D, dtype):
    g = torch.Generator().manual_seed(N + D)
    x = torch.randn(N, D, generator=g) * torch.exp(torch.randn(N, 1, generator=g) * 4)
    check_quantize(x.to(DTYPE[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_ties_borders_and_sentinels(dtype):
    x = torch.zeros(14, 96)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9375, 0.0])
    near = torch.cat((ties, ties * (1 + 2.0 ** -7), ties * (1 - 2.0 ** -7)))
    for n, e in enumerate((0, -126, 125, 7)):          # the ends of the scales' range among them
        x[n, 0] = 4.0
        x[n, 1:31], x[n, 32:62] = near, -near
        x[n, 31], x[n, 63] = -0.0, 4.0
        if e == 125:                                   # 7.9375 * 2^125 is finite
            x[n] = x[n].clamp(-7.9375, 7.9375)
        x[n] *= 2.0 ** e
    x[4, 40] = 1e-44                                   # a block of one subnormal
    x[5, 5], x[5, 40] = float("inf"), 1.0
    x[6, 70], x[6, 71] = float("nan"), 1.0
    x[7] = -3.0
    x[8, 7] = 3.3e38
    x[9] = torch.linspace(-1e-38, 1e-38, 96)
    x[10, 95] = float("-inf")
    x[11, :32] = torch.linspace(-2.0 ** -125, 2.0 ** -125, 32)
    x[12] = torch.randn(96) * 1e-37
    x[13] = -0.0
    check_quantize(x.to(DTYPE[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 3, 6])
def test_quantize_any_alignment_and_its_rows_only(dtype, offset):
    g = torch.Generator().manual_seed(offset)
    N, D = 3, 1001
    buf = torch.randn(N * D + offset, generator=g).to(DTYPE[dtype]).cuda()
    x = buf[offset:].view(N, D)
    raw = torch.full((N * D + 64,), 7.0, dtype=DTYPE[dtype], device="cuda")
    q = torch.full((N * 512 + 64,), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((N * 32 + 64,), 99, dtype=torch.uint8, device="cuda")
    sv.spec_mxfp4_quantize_rows(x, q[4:4 + N * 512].view(N, 512), s[4:4 + N * 32].view(N, 32),
                                raw[offset:offset + N * D].view(N, D))
    torch.cuda.synchronize()
    oq, os_, ov = ops.mxfp4_quantize(x.float().cpu().numpy())
    assert np.array_equal(q[4:4 + N * 512].view(N, 512).cpu().numpy(), oq)
    assert np.array_equal(s[4:4 + N * 32].view(N, 32).cpu().numpy(), os_)
    assert np.array_equal(raw[offset:offset + N * D].view(N, D).double().cpu().numpy(), ov)
    for t, n, lo in ((q, N * 512, 4), (s, N * 32, 4)):
        assert (t[:lo] == 99).all() and (t[lo + n:] == 99).all()
    assert (raw[:offset] == 7).all() and (raw[offset + N * D:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_in_the_place_of_x(dtype):
    x = torch.randn(50, 333).to(DTYPE[dtype]).cuda()
    oq, os_, ov = ops.mxfp4_quantize(x.float().cpu().numpy())
    q, s, _ = quantize(x, False)
    sv.spec_mxfp4_quantize_rows(x, q, s, x)
    torch.cuda.synchronize()
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_)
    assert np.array_equal(x.double().cpu().numpy(), ov)


# ------------------------------------------------------------------ product ---

def codes(n, D, seed, lo=115, hi=135):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (n, D // 2), generator=g).to(torch.uint8).cuda()
    s = torch.randint(lo, hi, (n, D // 32), generator=g).to(torch.uint8).cuda()
    return q, s


def product(a, sa, w, sw, dtype, out=None):
    out = torch.full((a.shape[0], w.shape[0]), 7.0, dtype=DTYPE[dtype], device="cuda") if out is None else out
    sv.spec_mxfp4_product(a, sa, w, sw, out)
    torch.cuda.synchronize()
    return out


def check_product(a, sa, w, sw, dtype, out):
    want, size = ops.mxfp4_product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    off = a.shape[1] * 2 / 64 * 2.0 ** -23 * size[fine]
    assert (np.abs(got - want)[fine] <= off + HALF[dtype] * (np.abs(want[fine]) + off)).all()


SHAPES = [(1, 128, 1), (1, 256, 8), (3, 128, 5), (1, 512, 4096), (16, 1024, 1000), (17, 384, 129), (33, 256, 127),
          (64, 512, 2056), (65, 4096, 300), (128, 128, 128), (130, 640, 513), (200, 2048, 1111), (256, 512, 4099),
          (300, 4096, 520), (513, 128, 260), (1000, 896, 777),
          # few rows: small tiles, at depths with two slots and with more
          (1, 4096, 300), (40, 4096, 999), (64, 4096, 1000), (33, 8192, 500), (7, 2176, 130), (32, 16384, 70),
          (64, 1024, 70001), (5, 256, 130001), (32, 4224, 9001),
          # the largest depth
          (2, 1 << 20, 33), (70, 1 << 20, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", SHAPES)
def test_product(N, D, V, dtype):
    print(f"\n[mxfp4 N={N} D={D} V={V} {dtype}]", flush=True)
    a, sa = codes(N, D, N + D)
    w, sw = codes(V, D, V + D + 1)
    check_product(a, sa, w, sw, dtype, product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [
    (33, 128, 51203), (64, 384, 51200), (65, 128, 57347), (128, 640, 57344), (129, 128, 28673), (300, 256, 28675),
    (257, 1152, 28672), (512, 2176, 14336),
    # several tiles for a workgroup of every tile, of one stage, two, three and five
    (3, 128, 90001), (20, 384, 85000), (32, 640, 82000), (5, 1152, 82003), (40, 128, 70001), (64, 384, 66000),
    (33, 640, 65700), (60, 1152, 65601), (70, 128, 70001), (128, 384, 66003), (100, 640, 66000), (66, 1152, 65700),
    (3, 2176, 40001), (20, 2432, 33300), (32, 2688, 33003), (5, 4096, 34000), (40, 2176, 33001), (64, 2432, 33300),
    (33, 2688, 33003), (60, 4096, 34000), (512, 128, 33000), (300, 384, 36001), (257, 640, 33003), (512, 1152, 32900),
])
def test_product_in_the_larger_tiles(N, D, V, dtype):
    print(f"\n[mxfp4 N={N} D={D} V={V} {dtype}]", flush=True)
    a, sa = codes(N, D, N + D)
    w, sw = codes(V, D, V + D + 1)
    check_product(a, sa, w, sw, dtype, product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 131), (35, 131), (64, 51203), (128, 57347), (300, 28675)])
def test_product_writes_its_rows_only(N, V, dtype):
    D = 128
    a, sa = codes(N, D, 3)
    w, sw = codes(V, D, 4)
    for offset in (0, 3):
        buf = torch.full((N * V + offset + 64,), 7.0, dtype=DTYPE[dtype], device="cuda")
        out = buf[offset:offset + N * V].view(N, V)
        product(a, sa, w, sw, dtype, out)
        check_product(a, sa, w, sw, dtype, out)
        assert (buf[:offset] == 7).all() and (buf[offset + N * V:] == 7).all()


@pytest.mark.parametrize("N", [1, 40, 300])
@pytest.mark.parametrize("lo,hi", [(60, 66), (150, 156), (0, 3)])
def test_product_of_small_and_large_scales(N, lo, hi):
    """Scales far from 1 on one side, their like on the other, so that products stay in range."""
    a, sa = codes(N, 256, 1, lo, hi)
    w, sw = codes(70, 256, 2, 254 - hi, 254 - lo)
    check_product(a, sa, w, sw, "f32", product(a, sa, w, sw, "f32"))


@pytest.mark.parametrize("N,V,D", [(5, 70, 256), (70, 300, 384), (300, 28675, 128)])
def test_product_of_blocks_that_stand_for_nan(N, V, D):
    a, sa = codes(N, D, 1)
    w, sw = codes(V, D, 2)
    sa[1, 0] = 255
    sa[N - 1, D // 32 - 1] = 255
    sw[3, 2] = 255
    a[1] = 0                                           # codes of zero change nothing
    out = product(a, sa, w, sw, "f32")
    check_product(a, sa, w, sw, "f32", out)
    assert torch.isnan(out[1]).all() and torch.isnan(out[:, 3]).all() and not torch.isnan(out[0, 0])


def test_product_past_32_bit_offsets():
    """Outputs and weights more than 2^32 bytes from their start."""
    N, D, V = 24, 128, 70_000_000
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 256, (V, D // 2), device="cuda", generator=g, dtype=torch.uint8)
    sw = torch.randint(120, 130, (V, D // 32), device="cuda", generator=g, dtype=torch.uint8)
    a, sa = codes(N, D, 5)
    out = product(a, sa, w, sw, "f32")
    for v in (0, 1 << 24, V - 300):
        check_product(a, sa, w[v:v + 300].contiguous(), sw[v:v + 300].contiguous(), "f32", out[:, v:v + 300].contiguous())
    del out, w
    torch.cuda.empty_cache()


def test_quantise_past_32_bit_offsets():
    N, D = 600_000, 4096                               # 4.9 GB of x
    x = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for n in range(0, N, 100_000):
        x[n:n + 100_000] = torch.randn(100_000, D, device="cuda", generator=g)
    q = torch.empty(N, D // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, D // 32, dtype=torch.uint8, device="cuda")
    sv.spec_mxfp4_quantize_rows(x, q, s)
    torch.cuda.synchronize()
    for n in (0, 524_280, N - 20):
        oq, os_, _ = ops.mxfp4_quantize(x[n:n + 20].float().cpu().numpy())
        assert np.array_equal(q[n:n + 20].cpu().numpy(), oq) and np.array_equal(s[n:n + 20].cpu().numpy(), os_)
    del x, q, s
    torch.cuda.empty_cache()


def test_quantised_product_is_near_the_real_one():
    """An entry of a block with largest magnitude A is off by at most A / 4 (saturation from just
    below 8 to 6 with a step of 2^e = at most A / 4; half a step of the top octave is no more)."""
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(20, 512, generator=g).cuda(), torch.randn(300, 512, generator=g).cuda()
    (qx, sx, _), (qw, sw, _) = quantize(x), quantize(w)
    got = product(qx, sx, qw, sw, "f32").double().cpu()
    xd, wd = x.double().cpu(), w.double().cpu()
    want = xd @ wd.t().contiguous()
    off = lambda t: (t.abs().view(t.shape[0], -1, 32).amax(2, keepdim=True) / 4).expand(-1, -1, 32).flatten(1)
    ox, ow = off(xd), off(wd)
    bound = xd.abs() @ ow.t().contiguous() + ox @ wd.abs().t().contiguous() + ox @ ow.t().contiguous()
    assert ((got - want).abs() <= bound * (1 + 1e-5)).all()


def test_quantise_and_product_replayed_from_a_graph():
    N, D, V = 33, 256, 1003
    x = torch.randn(N, D, device="cuda").to(torch.bfloat16)
    w, sw = codes(V, D, 7)
    q, s, _ = quantize(x, False)
    values = torch.empty_like(x)
    out = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")

    def step():
        sv.spec_mxfp4_quantize_rows(x, q, s, values)
        sv.spec_mxfp4_product(q, s, w, sw, out)

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
        oq, os_, ov = ops.mxfp4_quantize(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_)
        assert np.array_equal(values.double().cpu().numpy(), ov)
        check_product(q, s, w, sw, "bf16", out)
        eager = torch.empty_like(out)
        sv.spec_mxfp4_product(q, s, w, sw, eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def test_no_rows():
    e = lambda *shape, dtype=torch.uint8: torch.empty(*shape, dtype=dtype, device="cuda")
    sv.spec_mxfp4_quantize_rows(e(0, 40, dtype=torch.float32), e(0, 64), e(0, 4), e(0, 40, dtype=torch.float32))
    w, sw = codes(6, 128, 2)
    sv.spec_mxfp4_product(e(0, 64), e(0, 4), w, sw, e(0, 6, dtype=torch.float32))
    torch.cuda.synchronize()


def test_refusals_of_the_binding():
    a, sa = codes(4, 256, 1)
    w, sw = codes(6, 256, 2)
    out = torch.empty(4, 6, device="cuda")
    for bad in ((a.int(), sa, w, sw, out), (a, sa.float(), w, sw, out), (a, sa, w, sw, out.half())):
        with pytest.raises(TypeError):
            sv.spec_mxfp4_product(*bad)
    for bad in ((a, sa, w[:, :64].contiguous(), sw, out), (a, sa, w, sw[:3], out), (a, sa[:, :4].contiguous(), w, sw, out),
                (a, sa, w, sw, torch.empty(6, 4, device="cuda").t()), (a.cpu(), sa, w, sw, out)):
        with pytest.raises(ValueError):
            sv.spec_mxfp4_product(*bad)
    with pytest.raises(sv.SpecVerifyError):            # a depth that is no multiple of 128
        sv.spec_mxfp4_product(a[:, :32].contiguous(), sa[:, :2].contiguous(), w[:, :32].contiguous(),
                              sw[:, :2].contiguous(), out)
    with pytest.raises(sv.SpecVerifyError):            # rows that are not 16-byte aligned
        buf = torch.zeros(4 * 128 + 4, dtype=torch.uint8, device="cuda")
        sv.spec_mxfp4_product(buf[4:].view(4, 128), sa, w, sw, out)
    x = torch.randn(4, 200, device="cuda")
    q, s, v = quantize(x)
    with pytest.raises(TypeError):
        sv.spec_mxfp4_quantize_rows(x.half(), q, s)
    with pytest.raises(TypeError):
        sv.spec_mxfp4_quantize_rows(x, q, s, v.bfloat16())
    with pytest.raises(ValueError):                    # codes of unpadded rows
        sv.spec_mxfp4_quantize_rows(x, q[:, :100].contiguous(), s)
    with pytest.raises(sv.SpecVerifyError):            # values that overlap x, but are not x
        buf = torch.randn(4 * 200 + 8, device="cuda")
        sv.spec_mxfp4_quantize_rows(buf[:800].view(4, 200), q, s, buf[8:].view(4, 200))
