"""Host-side refusals of the grouped products (no GPU needed: arguments are checked before the device is touched)."""
import ctypes

from nvfp4_quantization_grouped_gb300 import gsa

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4
A = 0x10000
BIG = 1 << 40


def qin(data=A, scale=A, amax=A, data_bytes=BIG, scale_bytes=BIG >> 20):
    return gsa.QIn(data, scale, amax, data_bytes, scale_bytes)


def gemm(a=None, b=None, split=A, e=4, m=100, n=64, k=128, recipe=1, out=A, dtype=0):
    return gsa.load().gsa_grouped_gemm(a or qin(), b or qin(), split, e, m, n, k, recipe, out, dtype, None)


def test_product_refusals():
    assert gemm(e=0) == INVALID and gemm(m=-1) == INVALID and gemm(n=0) == INVALID and gemm(k=0) == INVALID
    assert gemm(recipe=2) == INVALID and gemm(dtype=1) == INVALID and gemm(dtype=3) == INVALID
    assert gemm(split=None) == INVALID and gemm(out=None) == INVALID
    assert gemm(a=qin(data=None)) == INVALID and gemm(b=qin(scale=None)) == INVALID
    assert gemm(a=qin(amax=None)) == INVALID and gemm(b=qin(amax=None)) == INVALID
    assert gemm(e=257) == UNSUP and gemm(k=96) == UNSUP and gemm(k=1 << 31) == UNSUP and gemm(m=1 << 31) == UNSUP
    assert gemm(n=1 << 30, e=4) == UNSUP
    assert gemm(a=qin(data=A + 8)) == ALIGN and gemm(b=qin(scale=A + 4)) == ALIGN and gemm(out=A + 8) == ALIGN
    assert gemm(split=A + 4) == ALIGN and gemm(a=qin(amax=A + 2)) == ALIGN
    assert gemm(a=qin(data_bytes=100 * 64 - 1)) == INVALID            # M K / 2 bytes of codes
    assert gemm(b=qin(data_bytes=4 * 64 * 64 - 1)) == INVALID
    assert gemm(b=qin(scale_bytes=4 * 1 * 2 * 512 - 1)) == INVALID    # E row tiles of 2 scale tiles
    assert gemm(a=qin(scale_bytes=2 * 512 - 1)) == INVALID
    assert gemm(m=0) == OK                                            # nothing to do
    L = gsa.load()
    assert L.gsa_grouped_gemm(None, ctypes.byref(qin()), A, 4, 10, 64, 128, 1, A, 0, None) == INVALID


def wgrad(a=None, b=None, split=A, e=4, m=100, n=64, k=128, recipe=1, out=A, dtype=2, acc=0, ws=A, ws_bytes=BIG):
    return gsa.load().gsa_grouped_gemm_wgrad(a or qin(), b or qin(), split, e, m, n, k, recipe, out, dtype, acc, ws,
                                             ws_bytes, None)


def test_weight_gradient_refusals():
    assert wgrad(e=0) == INVALID and wgrad(m=-1) == INVALID and wgrad(n=0) == INVALID and wgrad(k=0) == INVALID
    assert wgrad(recipe=7) == INVALID and wgrad(dtype=1) == INVALID and wgrad(split=None) == INVALID
    assert wgrad(out=None) == INVALID and wgrad(a=qin(data=None)) == INVALID and wgrad(b=qin(amax=None)) == INVALID
    assert wgrad(e=257) == UNSUP and wgrad(n=63) == UNSUP and wgrad(k=129) == UNSUP and wgrad(m=1 << 31) == UNSUP
    assert wgrad(n=1 << 30) == UNSUP
    assert wgrad(a=qin(scale=A + 4)) == ALIGN and wgrad(out=A + 4) == ALIGN and wgrad(ws=A + 128) == ALIGN
    assert wgrad(ws=None) == WS and wgrad(ws_bytes=100) == WS
    assert wgrad(n=1 << 29, k=1 << 29) == UNSUP                       # more tiles than counters hold


def test_weight_gradient_workspace():
    size = gsa.load().gsa_grouped_gemm_wgrad_workspace_size
    assert size(4, 100, 64, 128, 0) == 4 * 2 * 128                    # MXFP8: the tensor maps
    nv = size(4, 100, 64, 128, 1)
    # NVFP4: maps, tails (4 tiles a row tile), rows of (M + 15 E) / 2 + 8 E bytes on both sides
    assert nv >= 1024 + 2 * 4 * 4 * 512 + ((100 + 60) // 2 + 32) * (64 + 128) and nv % 256 == 0
    assert size(0, 100, 64, 128, 1) == 0 and size(257, 100, 64, 128, 1) == 0 and size(4, -1, 64, 128, 1) == 0
    assert size(4, 100, 64, 128, 2) == 0
