"""Refusals of the 4-bit operators' and the token scores' C entries, on the host before any HIP call
(no GPU needed: the pointers are never dereferenced); what their largest sizes enqueue; the streams
their binding takes."""
import ctypes

import pytest
import torch

import device_draft_verification_amd as sv
from test_draft_ops_dispatch import run, shim  # noqa: F401
from test_draft_ops_streams import Stream, two_devices  # noqa: F401

E, OK = sv.binding.SPEC_EINVAL, sv.binding.SPEC_OK


def P(at):
    return ctypes.c_void_p(at) if at is not None else None


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def quantize(lib, N=4, D=200, dtype=1, x=1 << 20, q=2 << 20, s=3 << 20, v=4 << 20):
    return lib.spec_mxfp4_quantize_rows(N, D, dtype, P(x), P(q), P(s), P(v), None)


def test_quantisation_refusals(lib):
    for bad in (dict(N=-1), dict(D=0), dict(D=-5), dict(dtype=2), dict(dtype=-1), dict(x=None), dict(q=None),
                dict(s=None), dict(x=(1 << 20) + 1), dict(q=(2 << 20) + 2), dict(s=(3 << 20) + 1),
                dict(v=(4 << 20) + 1), dict(dtype=0, x=(1 << 20) + 2), dict(dtype=0, v=(4 << 20) + 2),
                dict(v=(1 << 20) + 2), dict(v=(1 << 20) + 4 * 200 * 2 - 2), dict(v=(1 << 20) - 2),
                dict(N=1 << 28), dict(N=(1 << 31) - 1, D=1), dict(N=17, D=(1 << 31) - 200)):
        assert quantize(lib, **bad) == E, bad
    assert quantize(lib, N=0, x=None) == OK


def product(lib, N=4, D=256, V=70, a=1 << 20, sa=2 << 20, w=3 << 20, sw=4 << 20, dtype=1, out=5 << 20):
    return lib.spec_mxfp4_product(N, D, V, P(a), P(sa), P(w), P(sw), dtype, P(out), None)


def test_product_refusals(lib):
    for bad in (dict(N=-1), dict(V=0), dict(V=-1), dict(D=0), dict(D=64), dict(D=200), dict(D=-128),
                dict(D=sv.SPEC_MXFP4_MAX_DEPTH + 128), dict(dtype=2), dict(a=None), dict(sa=None), dict(w=None),
                dict(sw=None), dict(out=None), dict(a=(1 << 20) + 8), dict(w=(3 << 20) + 4), dict(sa=(2 << 20) + 2),
                dict(sw=(4 << 20) + 1), dict(out=(5 << 20) + 1), dict(dtype=0, out=(5 << 20) + 2),
                dict(N=(1 << 31) - 1, V=(1 << 31) - 1)):
        assert product(lib, **bad) == E, bad
    assert product(lib, N=0, a=None) == OK


def test_scores_refusals(lib):
    h = ctypes.c_void_p()
    good = [4, 1000, 20, 1]
    for at, bad in ((0, 0), (0, -1), (0, 1 << 24), (1, 0), (2, -1), (2, 65), (3, 2), (3, -1)):
        args = list(good)
        args[at] = bad
        assert lib.spec_logprobs_init(*args, None, ctypes.byref(h)) == E, (at, bad)
        assert not h.value
    assert lib.spec_logprobs_init(*good, None, None) == E
    p = P(1 << 20)
    assert lib.spec_token_logprobs(None, 1, p, p, None, p, p, p, p, p, p) == E
    assert lib.spec_token_logprobs_backward(None, 1, p, p, None, p, p, p, None, p) == E
    assert lib.spec_logprobs_set_stream(None, None) == E
    assert lib.spec_logprobs_destroy(None) == E


SCORES = r"""
import ctypes, json, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
shim.last_items.restype = ctypes.c_uint64
P = ctypes.c_void_p
A = [P((i + 1) << 52) for i in range(10)]
out = []
for rows, vocab, k, dtype, called in json.loads(sys.argv[3]):
    ctx = P()
    rc = [lib.spec_logprobs_init(rows, vocab, k, dtype, None, ctypes.byref(ctx))]
    seen = []
    if rc[0] == 0:
        n = shim.launch_count()
        rc.append(lib.spec_token_logprobs(ctx, called, *A[:9]))
        seen += [shim.launch_count() - n, shim.last_items()]
        n = shim.launch_count()
        rc.append(lib.spec_token_logprobs_backward(ctx, called, *A[:8]))
        seen += [shim.launch_count() - n, shim.last_items()]
        for bad in range(9):
            args = list(A[:9])
            if bad == 2:      # no temperatures: 1
                continue
            args[bad] = None
            rc.append(lib.spec_token_logprobs(ctx, called, *args))
            args[bad] = P(A[bad].value + 1)
            rc.append(lib.spec_token_logprobs(ctx, called, *args))
        rc.append(lib.spec_token_logprobs(ctx, rows + 1, *A[:9]))
        rc.append(lib.spec_token_logprobs(ctx, -1, *A[:9]))
        rc.append(lib.spec_token_logprobs_backward(ctx, rows + 1, *A[:8]))
        for bad in (0, 1, 3, 4, 5, 7):
            args = list(A[:8])
            args[bad] = None
            rc.append(lib.spec_token_logprobs_backward(ctx, called, *args))
            args[bad] = P(A[bad].value + 1)
            rc.append(lib.spec_token_logprobs_backward(ctx, called, *args))
        args = list(A[:8])
        args[7] = P(A[0].value + (4 if vocab * called > 4 else 1))   # overlaps the logits (or is misaligned)
        rc.append(lib.spec_token_logprobs_backward(ctx, called, *args))
        assert lib.spec_token_logprobs(ctx, 0, *[None] * 9) == 0
        lib.spec_logprobs_destroy(ctx)
    out.append((rc, seen))
print(json.dumps(out))
"""


def test_sizes_and_refusals_of_a_context(shim, monkeypatch):  # noqa: F811
    import test_draft_ops_dispatch as dispatch
    monkeypatch.setattr(dispatch, "CHILD", SCORES)
    most = (1 << 24) - 1
    calls = [(1, 152064, 64, 1, 1), (1, 1, 1, 0, 1), (4, 1 << 20, 64, 0, 3), (1023, 50000, 20, 1, 1023),
             (1024, 50000, 20, 1, 1024), (5000, 50000, 20, 1, 17), (most, 1000, 5, 1, most), (most, 5000, 64, 0, most),
             (1, (1 << 31) - 1, 64, 1, 1), (1, (1 << 31) - 1, 64, 0, 1)]
    for call, (rc, seen) in zip(calls, dispatch.run(shim, calls)):
        assert rc[:3] == [0, 0, 0], (call, rc)
        assert all(r == E for r in rc[3:]), (call, rc)
        assert seen[0] in (1, 2) and 0 < seen[1] < 1 << 32 and seen[2] == 1 and 0 < seen[3] < 1 << 32, (call, seen)


def test_products_and_quantisations_of_many_rows(shim):  # noqa: F811
    call = lambda n, d, v, t: ["spec_mxfp4_product", [n, d, v, "p0", "p1", "p2", "p3", t, "p4", None]]
    calls = [call(n, d, v, t) for n in (1, 33, 65, 129, 1 << 20) for d in (128, 4096) for v in (1, 152064) for t in (0, 1)]
    calls += [["spec_mxfp4_quantize_rows", [n, d, t, "p0", "p1", "p2", v, None]] for n, d in
              ((1, 1), (1, (1 << 31) - 200), (1 << 23, 2047), ((1 << 28) - 16, 1)) for t in (0, 1) for v in (None, "p3")]
    for c, (rc, n, items) in zip(calls, run(shim, calls)):
        assert rc == 0 and n == 1 and 0 < items < 1 << 32, (c, rc, n, items)
    # 2^23 tiles of rows: with 255 of the vocabulary a dispatch, with 256 too many
    for v, want in ((1 << 20, (OK, 1)), (255 * 256, (OK, 1)), (255 * 256 + 1, (E, 0))):
        n = 1 << 20 if v == 1 << 20 else (1 << 31) - 1
        for rc, launched, _ in run(shim, [call(n, 128, v, t) for t in (0, 1)]):
            assert (rc, launched) == want, (n, v)


def test_a_context_takes_streams_of_its_own_device_only(two_devices):  # noqa: F811
    lib, at = two_devices
    with pytest.raises(ValueError, match="spec_logprobs_init.*cuda:1"):
        sv.spec_logprobs_init(1, 100, 2, torch.float32, stream=Stream(1))
    assert lib.calls == []
    ctx = sv.spec_logprobs_init(1, 100, 2, torch.float32, stream=Stream(0))
    sv.spec_logprobs_set_stream(ctx, Stream(0))
    sv.spec_logprobs_set_stream(ctx)
    with pytest.raises(ValueError, match="spec_logprobs_set_stream.*cuda:1"):
        sv.spec_logprobs_set_stream(ctx, Stream(1))
    at.device = 1                       # the current stream is another device's
    with pytest.raises(ValueError, match="current device is cuda:1"):
        sv.spec_logprobs_set_stream(ctx)
    assert lib.calls == ["spec_logprobs_init"] + ["spec_logprobs_set_stream"] * 2
