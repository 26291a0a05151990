"""Host-side refusals of the gated products and of the products of unquantized rows (no GPU needed: arguments are checked
before the device is touched)."""
import ctypes
import math

from nvfp4_quantization_grouped_gb300 import gsa

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4
A = 0x10000
BIG = 1 << 40


def qin(data=A, scale=A, amax=A, data_bytes=BIG, scale_bytes=BIG >> 20):
    return gsa.QIn(data, scale, amax, data_bytes, scale_bytes)


def prm(limit=7.0, alpha=1.702, off=1.0):
    return gsa.ActParams(4.0, limit, alpha, off)


def common(call, groups=True):
    """What all four calls refuse alike."""
    assert call(e=0) == INVALID and call(m=-1) == INVALID and call(n=0) == INVALID and call(k=0) == INVALID
    assert call(recipe=2) == INVALID and call(dtype=3) == INVALID and call(dtype=-1) == INVALID
    assert call(split=None) == INVALID and call(b=qin(data=None)) == INVALID and call(b=qin(scale=None)) == INVALID
    assert call(b=qin(amax=None)) == INVALID
    assert call(e=257) == UNSUP and call(k=96) == UNSUP and call(k=1 << 31) == UNSUP and call(m=1 << 31) == UNSUP
    assert call(n=1 << 28, e=4) == UNSUP
    assert call(b=qin(data=A + 8)) == ALIGN and call(b=qin(scale=A + 4)) == ALIGN and call(split=A + 4) == ALIGN
    assert call(b=qin(amax=A + 2)) == ALIGN
    assert call(m=0) == OK
    if groups:
        assert call(groups=0) == INVALID and call(groups=3) == INVALID and call(n=64, groups=1) == UNSUP
        assert call(act=0) == INVALID and call(act=6) == INVALID and call(act=9) == INVALID
        assert call(act=3, params=None) == INVALID and call(act=3, params=prm(limit=0.0)) == INVALID
        assert call(act=3, params=prm(limit=math.inf)) == INVALID and call(act=3, params=prm(alpha=math.nan)) == INVALID
        assert call(act=3, params=prm(off=math.inf)) == INVALID
        assert call(probs=A + 2) == ALIGN
        # E * 2 N rows of K / 2 bytes; 2 E row tiles of 2 scale tiles
        assert call(b=qin(data_bytes=4 * 256 * 64 - 1)) == INVALID and call(b=qin(scale_bytes=8 * 2 * 512 - 1)) == INVALID


def glu(a=None, b=None, split=A, e=4, m=100, n=128, k=128, recipe=1, act=2, params=None, probs=A, groups=1, out=A, dtype=0):
    return gsa.load().gsa_grouped_glu(a or qin(), b or qin(), split, e, m, n, k, recipe, act, params, probs, groups, out, dtype, None)


def test_forward_refusals():
    common(glu)
    assert glu(out=None) == INVALID and glu(out=A + 8) == ALIGN and glu(dtype=1) == INVALID
    assert glu(a=qin(data=None)) == INVALID and glu(a=qin(amax=None)) == INVALID and glu(a=qin(data=A + 8)) == ALIGN
    assert glu(a=qin(data_bytes=100 * 64 - 1)) == INVALID and glu(a=qin(scale_bytes=2 * 512 - 1)) == INVALID
    assert gsa.load().gsa_grouped_glu(None, ctypes.byref(qin()), A, 4, 10, 128, 128, 1, 2, None, None, 1, A, 0, None) == INVALID


def bwd(dy=A, a=None, b=None, split=A, e=4, m=100, n=128, k=128, recipe=1, act=2, params=None, probs=A, groups=1, dx=A, dtype=0, dp=A, ws=A,
        ws_bytes=BIG):
    return gsa.load().gsa_grouped_glu_bwd(dy, a or qin(), b or qin(), split, e, m, n, k, recipe, act, params, probs, groups, dx, dtype, dp, ws,
                                          ws_bytes, None)


def test_gradient_refusals():
    common(bwd)
    assert bwd(dy=None) == INVALID and bwd(dx=None, dp=None) == INVALID and bwd(dtype=1) == INVALID
    assert bwd(dy=A + 8) == ALIGN and bwd(dx=A + 8) == ALIGN and bwd(dp=A + 2) == ALIGN and bwd(ws=A + 128) == ALIGN
    size = gsa.load().gsa_grouped_glu_bwd_workspace_size
    # the word of the split and four partial sums of a row for each 128 columns
    assert size(100, 128) == 256 + (4 * 100 * 4 + 255) // 256 * 256 and size(1, 129) == 256 + 256
    assert size(0, 128) == 0 and size(-1, 128) == 0 and size(5, 0) == 0 and size(1 << 31, 128) == 0
    assert bwd(ws_bytes=size(100, 128) - 1) == WS and bwd(ws=None) == WS


def gemv(x=A, xt=0, b=None, split=A, e=4, m=100, n=128, k=128, recipe=1, out=A, dtype=0, ws=A, ws_bytes=BIG):
    return gsa.load().gsa_grouped_gemv(x, xt, b or qin(), split, e, m, n, k, recipe, out, dtype, ws, ws_bytes, None)


def glu_gemv(x=A, xt=0, b=None, split=A, e=4, m=100, n=128, k=128, recipe=1, act=2, params=None, probs=A, groups=1, out=A, dtype=0,
             ws=A, ws_bytes=BIG):
    return gsa.load().gsa_grouped_glu_gemv(x, xt, b or qin(), split, e, m, n, k, recipe, act, params, probs, groups, out, dtype, ws, ws_bytes, None)


def test_products_of_unquantized_rows_refusals():
    common(gemv, False)
    common(glu_gemv)
    for call in (gemv, glu_gemv):
        assert call(x=None) == INVALID and call(out=None) == INVALID and call(xt=3) == INVALID and call(xt=-1) == INVALID
        assert call(x=A + 8) == ALIGN and call(out=A + 8) == ALIGN and call(ws=A + 128) == ALIGN
        assert call(ws=None) == WS and call(ws_bytes=100) == WS and call(m=1 << 28) == UNSUP and call(k=(1 << 30) + 64) == UNSUP
    size = gsa.load().gsa_grouped_gemv_workspace_size
    # 8 bytes a row, 8 rows of K / 2 bytes of codes each, scale tiles of 7 + 4 row tiles x 2
    assert size(4, 100, 128, 1) == 1024 + 800 * 64 + 11 * 2 * 512 and gemv(ws_bytes=size(4, 100, 128, 1) - 1) == WS
    assert size(0, 1, 64, 0) == 0 and size(257, 1, 64, 0) == 0 and size(1, 0, 64, 0) == 0 and size(1, 1, 32, 0) == 0 and size(1, 1, 64, 2) == 0
    assert gemv(b=qin(data_bytes=4 * 128 * 64 - 1)) == INVALID and gemv(b=qin(scale_bytes=4 * 2 * 512 - 1)) == INVALID
