"""gsa_moe_sort takes expert indices on any multiple of their size (no GPU needed: a missing workspace is found later)."""
from nvfp4_quantization_grouped_gb300 import gsa

A, ALIGN, WS = 0x10000, 3, 4


def test_index_alignment():
    def sort(idx, size):
        return gsa.load().gsa_moe_sort(idx, size, 100000, 1, 4, A, A, None, 0, None)

    assert [sort(A + i, 8) for i in (0, 8, 24)] == [WS] * 3
    assert [sort(A + i, 4) for i in (0, 4, 12, 20)] == [WS] * 4
    assert [sort(A + i, 8) for i in (1, 2, 4, 12)] == [ALIGN] * 4
    assert [sort(A + i, 4) for i in (1, 2, 6)] == [ALIGN] * 3
