"""A program asks gsa_version for the calls it needs: minor 2 has the expert-order calls and the grouped products."""
from nvfp4_quantization_grouped_gb300 import gsa


def test_version_says_which_calls_there_are():
    L = gsa.load()
    assert L.gsa_version() >= (1 << 16) | 2
    for name in gsa.EXPORTED:
        assert hasattr(L, name), name
