"""Refusals of the draft operators' C entries, on the host before any HIP call (no GPU needed:
the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import device_draft_verification_amd as sv

E, OK = sv.binding.SPEC_EINVAL, sv.binding.SPEC_OK


def P(at):
    return ctypes.c_void_p(at)


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_beam_init_refuses_bad_shapes(lib):
    h = ctypes.c_void_p()
    good = [4, 8, 8, 1000, 1]
    for at, bad in ((0, 0), (0, -1), (1, 0), (1, 65), (2, 0), (2, 65), (3, 0), (4, 2), (4, -1)):
        args = list(good)
        args[at] = bad
        assert lib.spec_beam_init(*args, None, ctypes.byref(h)) == E, (at, bad)
        assert not h.value
    assert lib.spec_beam_init(*good, None, None) == E
    # 2^24 rows of a row's pieces of 256 threads: the dispatch would pass 2^32 work-items
    assert lib.spec_beam_init(1 << 24, 1, 1, 1, 1, None, ctypes.byref(h)) == E
    assert lib.spec_beam_init((1 << 31) - 1, 64, 1, 1, 1, None, ctypes.byref(h)) == E
    assert lib.spec_beam_init(1, 1, 1, (1 << 31) - 1, 1, None, None) == E
    assert not h.value


def test_beam_calls_refuse_null(lib):
    assert lib.spec_beam_select(None, P(16), P(16), None, P(16), P(16), P(16), None) == E
    assert lib.spec_beam_set_stream(None, None) == E
    assert lib.spec_beam_destroy(None) == E


def reorder(lib, L=2, B=3, W=4, K=4, parent=0x100000, src=0x200000, ss=64, dst=0x400000, ds=64, n=64):
    return lib.spec_beam_reorder(L, B, W, K, P(parent), P(src), ss, P(dst), ds, n, None)


def test_reorder_refusals(lib):
    assert reorder(lib, L=-1) == E and reorder(lib, B=-1) == E
    assert reorder(lib, W=0) == E and reorder(lib, W=65) == E
    assert reorder(lib, K=0) == E and reorder(lib, K=65) == E
    assert reorder(lib, n=-1) == E
    assert reorder(lib, n=65) == E                       # strides below the bytes moved
    assert reorder(lib, ds=48) == E
    assert reorder(lib, parent=0x100002) == E            # misaligned parents
    assert lib.spec_beam_reorder(1, 1, 1, 1, None, P(16), 4, P(64), 4, 4, None) == E
    assert lib.spec_beam_reorder(1, 1, 1, 1, P(1 << 20), None, 4, P(64), 4, 4, None) == E
    assert lib.spec_beam_reorder(1, 1, 1, 1, P(1 << 20), P(16), 4, None, 4, 4, None) == E
    assert reorder(lib, dst=0x200000 + 64) == E          # overlapping ranges
    assert reorder(lib, dst=0x200000, K=3) == E          # the same place, other slots
    assert reorder(lib, dst=0x200000, ds=128) == E       # the same place, other strides
    assert reorder(lib, parent=0x200040) == E            # parents inside a state
    assert reorder(lib, parent=0x400000) == E
    assert reorder(lib, ss=1 << 61, ds=1 << 61) == E     # offsets past 63 bits
    assert reorder(lib, L=0) == OK and reorder(lib, B=0) == OK and reorder(lib, n=0) == OK


def distill(lib, which, rows=2, vocab=100, dtype=1, k=4, skip=None, odd=None):
    """One call with aligned stand-in pointers, `skip` replaced by NULL and `odd` misaligned."""
    names = {"forward": ["logits", "ids", "teacher", "tlse", "temp", "loss", "lse"],
             "backward": ["logits", "ids", "teacher", "tlse", "temp", "lse", "weight", "grad"],
             "loss_grad": ["logits", "ids", "teacher", "tlse", "temp", "weight", "loss", "lse", "grad"]}[which]
    at = {n: 0x1000000 * (i + 1) + (1 if n == odd else 0) for i, n in enumerate(names)}
    ptr = [None if n == skip else P(at[n]) for n in names]
    return getattr(lib, "spec_distill_" + which)(rows, vocab, dtype, k, *ptr, None), names


@pytest.mark.parametrize("which", ["forward", "backward", "loss_grad"])
def test_distill_refusals(lib, which):
    for bad in (dict(rows=-1), dict(vocab=0), dict(dtype=2), dict(k=0), dict(k=257), dict(rows=1 << 22)):
        assert distill(lib, which, **bad)[0] == E, bad
    assert distill(lib, which, rows=0)[0] == OK
    for name in distill(lib, which, rows=0)[1]:
        if name != "tlse":
            assert distill(lib, which, skip=name)[0] == E, name
        assert distill(lib, which, odd=name)[0] == E, name


def test_distill_refuses_a_gradient_across_the_logits(lib):
    p = [P(0x1000000 * (i + 1)) for i in range(9)]
    grad = P(0x1000000 + 100 * 2)  # the second row
    assert lib.spec_distill_loss_grad(2, 100, 1, 4, *p[:8], grad, None) == E
    assert lib.spec_distill_backward(2, 100, 1, 4, *p[:7], grad, None) == E


def test_int8_refusals(lib):
    x, q, s = P(0x100000), P(0x200000), P(0x300000)
    f = lib.spec_quantize_rows
    assert f(-1, 8, 1, x, q, s, None) == E and f(2, 0, 1, x, q, s, None) == E
    assert f(2, 8, 5, x, q, s, None) == E and f(1 << 24, 8, 1, x, q, s, None) == E
    assert f(2, 8, 1, None, q, s, None) == E and f(2, 8, 1, x, None, s, None) == E
    assert f(2, 8, 1, x, q, None, None) == E
    assert f(2, 8, 1, P(0x100001), q, s, None) == E and f(2, 8, 0, P(0x100002), q, s, None) == E
    assert f(2, 8, 1, x, q, P(0x300002), None) == E
    assert f(0, 8, 1, None, None, None, None) == OK
    g = lib.spec_int8_product
    p = [P(0x100000 * (i + 1)) for i in range(5)]
    ok = (2, 64, 100)
    assert g(-1, 64, 100, *p[:4], 1, p[4], None) == E
    for depth in (0, 8, 24, 131072):
        assert g(2, depth, 100, *p[:4], 1, p[4], None) == E, depth
    assert g(2, 64, 0, *p[:4], 1, p[4], None) == E
    assert g(*ok, *p[:4], 3, p[4], None) == E
    for i in range(4):
        bad = list(p[:4])
        bad[i] = None
        assert g(*ok, *bad, 1, p[4], None) == E
        bad[i] = P(0x100000 * (i + 1) + 2)
        assert g(*ok, *bad, 1, p[4], None) == E
    assert g(*ok, *p[:4], 1, None, None) == E
    assert g(*ok, *p[:4], 1, P(0x500001), None) == E and g(*ok, *p[:4], 0, P(0x500002), None) == E
    assert g(0, 64, 100, None, None, None, None, 1, None, None) == OK


def test_binding_checks_arguments_before_the_library():
    """Shapes, dtypes and devices are refused by the binding (CPU tensors here)."""
    f = torch.zeros
    with pytest.raises(ValueError):
        sv.spec_beam_reorder(f(2, 3, dtype=torch.int32), f(4, 5), f(4, 5))
    with pytest.raises((ValueError, TypeError)):
        sv.spec_distill_forward(f(2, 8), f(2, 3, dtype=torch.int64), f(2, 3), None, f(2), f(2), f(2).double())
    with pytest.raises(TypeError):
        sv.spec_distill_forward(f(2, 8).half(), f(2, 3, dtype=torch.int32), f(2, 3), None, f(2), f(2),
                                f(2).double())
    with pytest.raises(ValueError):
        sv.spec_quantize_rows(f(8), f(8, dtype=torch.int8), f(1))
    with pytest.raises(TypeError):
        sv.spec_quantize_rows(f(2, 8).double(), f(2, 8, dtype=torch.int8), f(2))
    with pytest.raises(ValueError):  # host tensors
        sv.spec_quantize_rows(f(2, 8), f(2, 8, dtype=torch.int8), f(2))
    with pytest.raises(ValueError):
        sv.spec_int8_product(f(2, 16, dtype=torch.int8), f(2), f(3, 16, dtype=torch.int8), f(3), f(2, 3))
