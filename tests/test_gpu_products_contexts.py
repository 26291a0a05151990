"""The grouped products in a second context of a device, in the first again, and in the device's next one after a reset: what the library has set up for a kernel, and
where the word for reports lies, are a context's own.  In a process of its own, whose contexts are made by hand."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

CODE = """
import ctypes, sys
sys.path[:0] = [ROOT, TESTS]
import numpy as np
from test_gpu_grouped_gemm import MX, NV, Matrices, padded
from nvfp4_quantization_grouped_gb300 import gsa
cu, L = ctypes.CDLL("libcuda.so.1"), gsa.load()
V = ctypes.c_void_p


def ok(r):
    assert r == 0, r


ok(cu.cuInit(0))
first, second, dev = V(), V(), ctypes.c_int()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(first), dev))
ok(cu.cuCtxCreate_v2(ctypes.byref(second), 0, dev))


class Buffers:   # of the current context
    def __init__(self):
        self.of = []

    def __call__(self, array):
        p = V()
        ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(max(256, array.nbytes))))
        ok(cu.cuMemcpyHtoD_v2(p, V(array.ctypes.data), ctypes.c_size_t(array.nbytes)))
        self.of.append(p)
        return p.value

    def back(self, at, like):
        out = np.empty_like(like)
        ok(cu.cuMemcpyDtoH_v2(V(out.ctypes.data), V(at), ctypes.c_size_t(out.nbytes)))
        return out

    def free(self):
        for p in self.of:
            ok(cu.cuMemFree_v2(p))


def calls(recipe, rows):
    rng = np.random.default_rng(rows)
    n, k, split, m = 128, 128, [rows, 3], rows + 3
    to, e = Buffers(), 2
    mp = padded(split, recipe)
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [2 * n] * e, k, recipe)
    ca, cb = Matrices(rng, [n] * e, mp, recipe), Matrices(rng, [k] * e, mp, recipe)
    qin = lambda q: gsa.QIn(to(q.data), to(q.scale), to(q.amax), q.data.size - 1, q.scale.size)
    qa, qb, qca, qcb = qin(a), qin(b), qin(ca), qin(cb)
    s, bad = to(np.array(split, np.int64)), to(np.array([rows, 4], np.int64))
    dy = to(rng.integers(0x3F00, 0x4000, (m, n), dtype=np.uint16))
    x = to(rng.standard_normal((m, k)).astype(np.float32))
    ws = to(np.zeros(1 << 25, np.uint8))
    assert ws % 256 == 0
    shape = (e, m, n, k, recipe)
    wide = (e, m, 2 * n, k, recipe)
    of = {"product": ((m, 2 * n), lambda sp, o: L.gsa_grouped_gemm(qa, qb, sp, *wide, o, gsa.FP32, None)),
          "gradient": ((e, n, k), lambda sp, o: L.gsa_grouped_gemm_wgrad(qca, qcb, sp, *shape, o, gsa.FP32, 0, ws, 1 << 25, None)),
          "gated": ((m, n), lambda sp, o: L.gsa_grouped_glu(qa, qb, sp, *shape, 2, None, None, 1, o, gsa.FP32, None)),
          "gated gradient": ((m, 2 * n), lambda sp, o: L.gsa_grouped_glu_bwd(dy, qa, qb, sp, *shape, 2, None, None, 1, o, gsa.FP32, to(np.zeros(m, np.float32)),
                                                                             ws, 1 << 25, None)),
          "rows": ((m, 2 * n), lambda sp, o: L.gsa_grouped_gemv(x, gsa.FP32, qb, sp, *wide, o, gsa.FP32, ws, 1 << 25, None)),
          "gated rows": ((m, n), lambda sp, o: L.gsa_grouped_glu_gemv(x, gsa.FP32, qb, sp, *shape, 2, None, None, 1, o, gsa.FP32, ws, 1 << 25, None))}
    out = {}
    for name, (size, call) in of.items():
        like = np.full(size, 7.0, np.float32)
        o, kept = to(like), to(like)
        assert call(s, o) == 0, name
        assert L.gsa_grouped_gemm_status(None) == 0, name
        out[name] = to.back(o, like)
        assert np.isfinite(out[name]).all() and not (out[name] == 7.0).all(), name
        assert call(bad, kept) == 0 and L.gsa_grouped_gemm_status(None) == 1 and L.gsa_grouped_gemm_status(None) == 0, name
        assert (to.back(kept, like) == 7.0).all(), name
    to.free()
    return out


seen = {}
for context in (first, second, first, second):
    ok(cu.cuCtxSetCurrent(context))
    for recipe in (MX, NV):
        for rows in (10, 20000):   # single blocks, pairs
            for name, v in calls(recipe, rows).items():
                assert np.array_equal(seen.setdefault((recipe, rows, name), v), v), name
ok(cu.cuCtxSynchronize())
ok(cu.cuCtxDestroy_v2(second))
ok(cu.cuDevicePrimaryCtxReset_v2(dev))   # this process's own
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(first), dev))
ok(cu.cuCtxSetCurrent(first))
for recipe in (MX, NV):
    for rows in (10, 20000):
        for name, v in calls(recipe, rows).items():
            assert np.array_equal(seen[(recipe, rows, name)], v), name
print("same", len(seen))
"""


def test_two_contexts():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = CODE.replace("ROOT", repr(os.path.dirname(tests))).replace("TESTS", repr(tests))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same", "24"], r.stdout + r.stderr
