"""The gated products' and the unquantized rows' helpers launch on the current device: tensors or a stream of another one are
refused before the library is called.  No GPU needed (stand-ins for tensors)."""
import pytest
import torch

from test_moe_devices import BF16, F32, HERE, I64, THERE, U8, Library, Stream, Tensor, lib  # noqa: F401

from nvfp4_quantization_grouped_gb300 import gsa


class Sized(Tensor):
    def numel(self):
        return self.shape.numel()


def calls(dev, stream=None, other=None):
    """name -> one call with all of its tensors on dev (probs on `other`, where given)."""
    def t(dtype, *shape):
        return Sized(dev, dtype, *shape)

    q = {"row_data": t(U8, 1 << 20), "row_scale": t(U8, 1 << 20)}
    split, x, y, probs = t(I64, 2), t(BF16, 8, 64), t(BF16, 8, 128), Sized(other or dev, F32, 8)
    return {
        "gsa_grouped_glu": lambda: gsa.grouped_glu(q, q, split, 8, 128, 64, gsa.MXFP8, probs=probs, out=y, stream=stream),
        "gsa_grouped_glu_bwd": lambda: gsa.grouped_glu_bwd(y, q, q, split, 8, 128, 64, gsa.MXFP8, probs=probs, want_dprobs=False,
                                                           out=(t(BF16, 8, 256), None), stream=stream),
        "gsa_grouped_gemv": lambda: gsa.grouped_gemv(x, q, split, 128, gsa.MXFP8, out=y if other is None else Sized(other, BF16, 8, 128)),
        "gsa_grouped_glu_gemv": lambda: gsa.grouped_glu_gemv(x, q, split, 128, gsa.MXFP8, probs=probs, out=y)}


NAMES = sorted(calls(HERE))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_the_current_device_are_taken(lib, name):  # noqa: F811
    calls(HERE)[name]()
    assert [c for c in lib.calls if not c.endswith("size")] == [name]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(lib, name):  # noqa: F811
    with pytest.raises(gsa.GsaError, match="current device"):
        calls(THERE)[name]()
    with pytest.raises(gsa.GsaError):
        calls(HERE, other=THERE)[name]()
    assert [c for c in lib.calls if not c.endswith("size")] == []


@pytest.mark.parametrize("name", ["gsa_grouped_glu", "gsa_grouped_glu_bwd"])
def test_a_stream_of_another_device_is_refused(lib, name):  # noqa: F811
    with pytest.raises(gsa.GsaError, match="stream of cuda:1"):
        calls(HERE, Stream(THERE))[name]()
    assert [c for c in lib.calls if not c.endswith("size")] == []
