"""The score kernels' own source run on the host (no GPU), their wavefronts in given orders: between
two barriers one wavefront runs as far as it can before the next begins (tests/wavefronts), and so
does a lane between two exchanges. Rows must come out the same in every order, without a wavefront
that waits where others do not."""
import ctypes
import glob
import itertools
import multiprocessing
import os
import subprocess

import numpy as np
import pytest

from oracle import draft_ops as ops

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "device_draft_verification_amd", "csrc")
CLANG = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "clang++")

# What a host compiler does not know: a launch, and instructions in their own language.
REPLACED = {
    "launch.hpp": [("kern<<<grid, block, shmem, stream>>>(args...)", "kern(args...)")],
    "logprobs.hip": [
        ('asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));', "r = fmaxf(fmaxf(a, b), c);"),
        ('asm("v_maximum3_f32 %0, %1, %2, %2" : "=v"(r) : "v"(a), "v"(b));',
         "r = a != a ? a : b != b ? b : fmaxf(a, b);")],
}
HOST_PART = "bool aligned(const void* p, size_t a)"     # from here on the source is the host's

fork = multiprocessing.get_context("fork")

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG), reason="needs clang's vector types")


def device_source(name, text):
    for old, new in REPLACED.get(name, []):
        assert text.count(old) == 1, (name, old)
        text = text.replace(old, new)
    return text


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("wavefronts")
    for path in glob.glob(os.path.join(CSRC, "*.hpp")):
        name = os.path.basename(path)
        (d / name).write_text(device_source(name, open(path).read()))
    text = device_source("logprobs.hip", open(os.path.join(CSRC, "logprobs.hip")).read())
    assert text.count(HOST_PART) == 1
    text = text.split(HOST_PART)[0] + "}  // namespace\n}  // namespace specv\n"
    src, out = d / "scores.cpp", d / "scores.so"
    src.write_text(text + open(os.path.join(HERE, "wavefronts", "scores.cpp")).read())
    subprocess.run([CLANG, "-std=c++17", "-O1", "-ffp-contract=off", "-w", "-fPIC", "-shared", "-I",
                    os.path.join(HERE, "wavefronts"), "-I", str(d), "-I", os.path.join(ROOT, "include"), "-o", str(out),
                    str(src)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.run_scores.restype = ctypes.c_char_p
    return lib


def bf16(z):
    """Rounded to bf16: as 16-bit words, and as binary32 values."""
    b = z.astype(np.float32).view(np.uint32)
    w = ((b + 0x7FFF + (b >> 16 & 1)) >> 16).astype(np.uint16)
    return w, (w.astype(np.uint32) << 16).view(np.float32)


def scores(lib, z, token, keep, order, splits=1, dtype="bf16"):
    """(fault, outputs, the logits as binary32)."""
    N, V = z.shape
    data, values = bf16(z) if dtype == "bf16" else (z.astype(np.float32), z.astype(np.float32))
    raw = np.zeros(data.nbytes + 64, np.uint8)                  # 16-byte aligned, with room behind
    at = -raw.ctypes.data % 16
    raw[at:at + data.nbytes] = data.reshape(-1).view(np.uint8)
    groups = V // (8 if dtype == "bf16" else 4) + 2
    per = (-(-groups // splits) + 7) // 8 * 8
    f = lambda *s: np.full(s, 7, np.float32)
    i = lambda *s: np.full(s, 77, np.int32)
    out = dict(logprob=f(N), rank=i(N), entropy=f(N), top_token=i(N, keep), top_logprob=f(N, keep), norm=f(N, 2))
    P = ctypes.c_void_p
    token, order = np.ascontiguousarray(token, np.int32), np.asarray(order, np.int32)

    def call(to):
        fault = lib.run_scores(1 if dtype == "bf16" else 0, int(keep > 0), N, V, keep, splits, per, P(order.ctypes.data),
                               P(raw.ctypes.data + at), P(token.ctypes.data), None,
                               *[P(x.ctypes.data) for x in out.values()])
        to.send((fault, out))

    # in a process of its own: wavefronts that disagree may leave their arrays
    here, there = fork.Pipe(duplex=False)
    child = fork.Process(target=call, args=(there,))
    child.start()
    there.close()
    try:
        fault, out = here.recv()
    except EOFError:
        fault = b"the process ended"
    child.join()
    return fault, out, values


def check(got, values, token, keep):
    want = ops.token_scores(values, token, None, keep)
    assert np.array_equal(got["rank"], want["rank"]) and np.array_equal(got["top_token"], want["top_token"])
    # Sums as in tests/test_gpu_logprobs.py, the host's exponentials within a step as well
    D = 2.0 ** -23 * (np.log(values.shape[1]) + 6)
    for k in ("logprob", "top_logprob", "norm"):
        fine = np.isfinite(want[k])
        assert np.array_equal(got[k][~fine], want[k][~fine], equal_nan=True)
        assert (np.abs(got[k][fine] - want[k][fine]) <= D + 2.0 ** -24 * np.abs(want[k][fine])).all()


ORDERS = [(0, 1, 2, 3), (3, 2, 1, 0), (1, 3, 0, 2), (2, 0, 3, 1)]


def rows(kind, V, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal(V) * 2.5
    if kind == "rising":       # every segment overflows the list: it is gone through again
        z = np.arange(V) / 1000.0
    elif kind == "levels":     # lists of equal entries are ranked
        z = np.where(np.arange(V) % 5 == 2, 1.0, 0.0)
    elif kind == "late":
        z = np.where(np.arange(V) >= V - 700, 5.0, -5.0) + np.arange(V) / 40000
    elif kind == "uneven":     # only one wavefront's groups hold what the lists keep
        z = z + np.where(np.arange(V) // 512 % 4 == seed % 4, 20.0, 0.0)
    return z[None].astype(np.float32)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("V,dtype", [(5, "bf16"), (700, "f32"), (2048, "bf16"), (4099, "f32"), (8200, "bf16")])
def test_rows_of_one_segment(lib, V, dtype, order):
    """Groups that a wavefront puts aside are read by other lanes than wrote them."""
    for keep, seed in ((8, 1), (64, 2)):
        z = rows("normal", V, seed)
        fault, got, values = scores(lib, z, [V // 3], keep, order, dtype=dtype)
        assert fault is None, (fault, V, keep, order)
        check(got, values, [V // 3], keep)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("kind", ["normal", "rising", "levels", "late", "uneven"])
def test_rows_of_several_segments(lib, kind, order):
    V = 41003                                            # segments of 1, 3 and 2 steps
    for keep, seed in ((20, 1), (64, 2), (1, 3)):
        z = rows(kind, V, seed)
        token = [int(np.argmax(z))] if seed == 1 else [V // 2]
        fault, got, values = scores(lib, z, token, keep, order)
        assert fault is None, (fault, kind, keep, order)
        check(got, values, token, keep)


@pytest.mark.parametrize("order", ORDERS)
def test_rows_in_parts(lib, order):
    V = 41003
    z, token = rows("normal", V, 5), [17]
    for splits, keep, dtype in ((2, 20, "f32"), (5, 64, "bf16")):
        fault, got, values = scores(lib, z, token, keep, order, splits, dtype)
        assert fault is None, (fault, splits, order)
        check(got, values, token, keep)


def test_any_order_gives_the_same_list(lib):
    """Entries that many segments keep, every order of the four wavefronts."""
    V = 26000
    z = rows("normal", V, 9)
    for order in itertools.permutations(range(4)):
        fault, got, values = scores(lib, z, [3], 8, order)
        assert fault is None, (fault, order)
        check(got, values, [3], 8)
