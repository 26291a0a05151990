"""Host-side refusals of the gsa_moe_* calls (no GPU needed: arguments are
checked before the device is touched)."""
from nvfp4_quantization_grouped_gb300 import gsa

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4
A = 0x10000


def test_sort_refusals():
    L = gsa.load()

    def sort(idx=A, b=8, t=10, k=2, e=4, row=A, split=A, ws=None, n=0):
        return L.gsa_moe_sort(idx, b, t, k, e, row, split, ws, n, None)

    assert sort(b=2) == INVALID and sort(t=-1) == INVALID and sort(k=0) == INVALID and sort(e=0) == INVALID
    assert sort(idx=None) == INVALID and sort(row=None) == INVALID and sort(split=None) == INVALID
    assert sort(e=257) == UNSUP and sort(t=1 << 30, k=2) == UNSUP and sort(t=1 << 40, k=1 << 40) == UNSUP
    assert sort(idx=A + 4) == ALIGN and sort(row=A + 4) == ALIGN and sort(split=A + 4) == ALIGN
    assert sort(t=100000) == WS and sort(t=100000, ws=A, n=16) == WS
    assert L.gsa_moe_sort_workspace_size(16, 8, 128) == 0
    need = L.gsa_moe_sort_workspace_size(100000, 2, 4)
    assert need > 0 and need % 16 == 0
    assert L.gsa_moe_sort_workspace_size(100000, 2, 257) == 0


def test_row_call_refusals():
    L = gsa.load()
    calls = {
        "permute": lambda x=A, p=A, row=A, t=4, k=2, h=64, d=0, y=A, q=A: L.gsa_moe_permute(x, p, row, t, k, h, d, y, q,
                                                                                             None),
        "permute_bwd": lambda x=A, p=A, row=A, t=4, k=2, h=64, d=0, y=A, q=A: L.gsa_moe_permute_bwd(x, p, row, t, k, h,
                                                                                                    d, y, q, None),
        "unpermute": lambda x=A, p=A, row=A, t=4, k=2, h=64, d=0, y=A, q=A: L.gsa_moe_unpermute(x, p, row, t, k, h, d,
                                                                                                y, None),
        "unpermute_bwd": lambda x=A, p=A, row=A, t=4, k=2, h=64, d=0, y=A, q=A: L.gsa_moe_unpermute_bwd(
            x, A, p, row, t, k, h, d, y, q, None)}
    for name, f in calls.items():
        assert f(t=-1) == INVALID and f(k=0) == INVALID and f(h=0) == INVALID and f(d=3) == INVALID, name
        assert f(x=None) == INVALID and f(row=None) == INVALID, name
        assert f(t=1 << 30) == UNSUP and f(h=1 << 31) == UNSUP, name
        assert f(x=A + 8) == ALIGN and f(y=A + 2) == ALIGN and f(row=A + 2) == ALIGN and f(p=A + 2) == ALIGN, name
        if name != "unpermute_bwd":
            assert f(y=None) == INVALID, name
    assert calls["permute"](q=None) == INVALID and calls["permute"](p=None) == INVALID
    assert calls["permute_bwd"](q=None) == INVALID
    assert calls["unpermute_bwd"](y=None, q=None) == INVALID
    assert L.gsa_moe_unpermute_bwd(A, None, A, A, 4, 2, 64, 0, A, A, None) == INVALID   # dweights need ys
