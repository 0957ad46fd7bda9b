"""What the draft operators' C entries enqueue at their largest sizes, on the host (no GPU): a small
library in front of the HIP runtime takes the launches and keeps their sizes. One dispatch holds
fewer than 2^32 work-items; the runtime refuses a larger one, so a call whose arguments pass the
checks must not come to it."""
import json
import os
import subprocess
import sys

import pytest

import device_draft_verification_amd as sv

SHIM = r"""
#include <stdint.h>
typedef struct { uint32_t x, y, z; } size3;
static uint64_t items;
static int launches;
int hipLaunchKernel(const void *f, size3 g, size3 b, void **args, unsigned long lds, void *stream) {
    items = (uint64_t)g.x * g.y * g.z * b.x * b.y * b.z;
    ++launches;
    return 0;
}
static size3 grid, block;
int __hipPushCallConfiguration(size3 g, size3 b, unsigned long lds, void *stream) {
    grid = g;
    block = b;
    return 0;
}
int __hipPopCallConfiguration(size3 *g, size3 *b, unsigned long *lds, void **stream) {
    *g = grid;
    *b = block;
    *lds = 0;
    *stream = 0;
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipMalloc(void **p, unsigned long n) { *p = (void *)0x10000000; return 0; }
int hipFree(void *p) { return 0; }
int hipStreamSynchronize(void *s) { return 0; }
uint64_t last_items(void) { return items; }
int launch_count(void) { return launches; }
"""

CHILD = r"""
import ctypes, json, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
shim.last_items.restype = ctypes.c_uint64
P, I = ctypes.c_void_p, ctypes.c_longlong
A = [P((i + 1) << 52) for i in range(10)]      # aligned, far apart, never looked at
out = []
for name, args in json.loads(sys.argv[3]):
    before = shim.launch_count()
    if name == "spec_beam_select":
        ctx = P()
        rc = lib.spec_beam_init(*args, None, ctypes.byref(ctx))
        if rc == 0:
            rc = lib.spec_beam_select(ctx, A[0], A[1], None, *A[2:6])
            lib.spec_beam_destroy(ctx)
    else:
        f = getattr(lib, name)
        rc = f(*[A[int(a[1:])] if isinstance(a, str) else None if a is None else I(a) for a in args])
    out.append((rc, shim.launch_count() - before, shim.last_items()))
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("shim")
    src, lib = d / "shim.c", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(lib), str(src)], check=True)
    return str(lib)


def run(shim, calls):
    r = subprocess.run([sys.executable, "-c", CHILD, shim, sv.binding.LIB_PATH, json.dumps(calls)],
                       capture_output=True, text=True, timeout=120, env=dict(os.environ))
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout)


def enqueued(shim, calls, launches=1):
    for call, (rc, n, items) in zip(calls, run(shim, calls)):
        assert rc == 0 and n == launches and 0 < items < 1 << 32, (call, rc, n, items)


def refused(shim, calls):
    for call, (rc, n, _) in zip(calls, run(shim, calls)):
        assert rc == sv.binding.SPEC_EINVAL and n == 0, (call, rc, n)


def test_quantisation_of_many_rows(shim):
    rows = (1, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, (1 << 24) - 1)
    cols = (1, 512, 1024, 1032, 2048, 2056, 4096, 4104, 8184, 8192, 8200, 16384, 20000)
    call = lambda n, d, t: ["spec_quantize_rows", [n, d, t, "p0", "p1", "p2", None]]
    enqueued(shim, [call(n, d, t) for n in rows for d in cols for t in (0, 1)])
    refused(shim, [call(1 << 24, d, t) for d in cols for t in (0, 1)])


def test_distillation_of_many_rows(shim):
    p = [f"p{i}" for i in range(9)]
    calls = [(n, v, t, k) for n in (1, 256, 257, (1 << 22) - 1) for v in (1, 5000, 152064, (1 << 31) - 1)
             for t in (0, 1) for k in (1, 256)]
    for name, count in (("forward", 7), ("backward", 8), ("loss_grad", 9)):
        enqueued(shim, [["spec_distill_" + name, [n, v, t, k, *p[:count], None]] for n, v, t, k in calls
                        if not (n * v > 1 << 50)])


def test_product_of_many_rows(shim):
    call = lambda n, d, v, t: ["spec_int8_product", [n, d, v, "p0", "p1", "p2", "p3", t, "p4", None]]
    enqueued(shim, [call(n, d, v, t) for n in (1, 33, 65, 129, 1 << 20) for d in (16, 4096)
                    for v in (1, 152064) for t in (0, 1)])
    # 2^40 outputs: more tiles than one dispatch holds
    refused(shim, [call(1 << 20, 16, 1 << 20, t) for t in (0, 1)])


def test_reordering_of_many_states(shim):
    call = lambda L, B, n, same: ["spec_beam_reorder", [L, B, 64, 64, "p0", "p1", n, "p1" if same else "p2", n, n, None]]
    enqueued(shim, [call(L, B, n, same) for L, B in ((1, 1), (64, 4096)) for n in (1, 4, 16, 1 << 20)
                    for same in (False, True)])


def test_selection_of_many_beams(shim):
    # batch, beams, keep, vocab, dtype; two kernels, the second's size seen
    enqueued(shim, [["spec_beam_select", [b, w, k, v, t]] for b, w, v in
                    ((1, 1, 1), (4096, 64, 152064), ((1 << 18) - 1, 64, 8), (1, 64, 1 << 22)) for k in (1, 64)
                    for t in (0, 1)], launches=2)
    refused(shim, [["spec_beam_select", [1 << 24, 1, 1, 8, 1]]])
