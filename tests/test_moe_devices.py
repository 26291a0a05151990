"""The moe_* and grouped_* helpers launch on the current device, so tensors (or a stream) of another device are refused
before the library is called.  No GPU needed: stand-ins for tensors say where they are."""
import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

HERE, THERE = torch.device("cuda", 0), torch.device("cuda", 1)
U8, I32, I64, F32, BF16 = torch.uint8, torch.int32, torch.int64, torch.float32, torch.bfloat16


class Tensor:
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        self.device, self.dtype, self.shape = device, dtype, torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        pass


class Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device = device


class Library:
    """Counts the calls that would launch."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 0
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    if gsa._torch is None:
        gsa._setup()
    lib = Library()
    monkeypatch.setattr(gsa, "_lib", lib)
    monkeypatch.setattr(gsa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(gsa, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(device, dtype, *shape))
    return lib


def calls(dev, stream=None):
    """name -> one call of each helper with all of its tensors on dev."""
    def t(dtype, *shape):
        return Tensor(dev, dtype, *shape)

    row, x, big = t(I32, 4, 2), t(BF16, 4, 64), t(BF16, 8, 64)
    q = {s + "_" + k: v for s in ("row", "col") for k, v in (("data", t(U8, 4096)), ("scale", t(U8, 4096)))}
    split = t(I64, 2)
    return {
        "gsa_moe_sort": lambda: gsa.moe_sort(t(I64, 4, 2), 3, (row, t(I64, 4)), stream=stream),
        "gsa_moe_permute": lambda: gsa.moe_permute(x, row, out=big, stream=stream),
        "gsa_moe_permute_bwd": lambda: gsa.moe_permute_bwd(big, row, out=x, stream=stream),
        "gsa_moe_unpermute": lambda: gsa.moe_unpermute(big, row, out=x, stream=stream),
        "gsa_moe_unpermute_bwd": lambda: gsa.moe_unpermute_bwd(x, big, row, out=(big, t(F32, 4, 2)), stream=stream),
        "gsa_grouped_gemm": lambda: gsa.grouped_gemm(q, q, split, 8, 64, 64, gsa.MXFP8, out=t(F32, 8, 64), stream=stream),
        "gsa_grouped_gemm_wgrad": lambda: gsa.grouped_gemm_wgrad(q, q, split, 8, 64, 64, gsa.MXFP8, out=t(F32, 2, 64, 64),
                                                                 accumulate=True)}


NAMES = sorted(calls(HERE))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_the_current_device_are_taken(lib, name):
    calls(HERE)[name]()
    assert lib.calls == [name]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(lib, name):
    with pytest.raises(gsa.GsaError, match="current device"):
        calls(THERE)[name]()
    assert lib.calls == []


@pytest.mark.parametrize("name", [n for n in NAMES if n != "gsa_grouped_gemm_wgrad"])
def test_a_stream_of_another_device_is_refused(lib, name):
    calls(HERE, Stream(HERE))[name]()
    with pytest.raises(gsa.GsaError, match="stream of cuda:1"):
        calls(HERE, Stream(THERE))[name]()
    assert lib.calls == [name]
