"""The weight gradient's tensor maps, which its first kernel writes into the workspace and its second reads: the same
results whatever the workspace held before, call after call and on two streams at once, and no memory touched behind the
operands."""
import ctypes
import mmap

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split, padded

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

# even pitches, odd ones (NVFP4 copies those rows), empty experts; narrow sides (single blocks) and wide (pairs)
SHAPES = [([0, 0, 128, 1, 127, 129, 0], 128, 130), ([256, 512], 128, 256), ([300, 17, 0, 64], 320, 512),
          ([33, 97, 64, 1, 32] * 8, 64, 96), ([2000, 16, 0, 48], 256, 384)]


class Call:
    """One weight gradient on buffers of its own, with any workspace and stream, through the C entry point."""

    def __init__(self, rng, split, n, k, recipe):
        mp = padded(split, recipe)
        self.a, self.b = (Matrices(rng, [w] * len(split), mp, recipe) for w in (n, k))
        self.qa, self.qb, self.split = self.a.dev("col"), self.b.dev("col"), dev_split(split)
        self.args = (len(split), sum(split), n, k, recipe)
        self.ref = np.stack([x @ w.T for x, w in zip(self.a.values, self.b.values)])
        self.nbytes = gsa.load().gsa_grouped_gemm_wgrad_workspace_size(*self.args)
        self.dw = torch.empty((len(split), n, k), device="cuda")

    def __call__(self, ws, stream):
        qa, qb = (gsa.QIn(q["col_data"].data_ptr(), q["col_scale"].data_ptr(), q["amax_col"].data_ptr(),
                          q["col_data"].numel(), q["col_scale"].numel()) for q in (self.qa, self.qb))
        return gsa.load().gsa_grouped_gemm_wgrad(ctypes.byref(qa), ctypes.byref(qb), self.split.data_ptr(), *self.args,
                                                 self.dw.data_ptr(), gsa.FP32, 0, ws.data_ptr(), self.nbytes,
                                                 stream.cuda_stream)

    def right(self):
        return np.array_equal(self.dw.double().cpu().numpy(), self.ref)


def calls(recipe):
    rng = np.random.default_rng(31)
    return [Call(rng, *s, recipe) for s in SHAPES]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("fill", [0xFF, 0x5A])
def test_one_workspace_for_calls_of_many_shapes(recipe, fill):
    cs, s = calls(recipe), torch.cuda.current_stream()
    ws = torch.empty(max(c.nbytes for c in cs), dtype=torch.uint8, device="cuda")
    for _ in range(100):
        for c in cs:
            c.dw.fill_(float("nan"))
            ws.fill_(fill)
            assert c(ws, s) == 0
    assert gsa.grouped_gemm_status() == 0
    assert all(c.right() for c in cs)
    for c in cs:      # back to back, every call's maps where another call's were
        c.dw.fill_(float("nan"))
    for _ in range(100):
        for c in cs:
            assert c(ws, s) == 0
    assert gsa.grouped_gemm_status() == 0
    assert all(c.right() for c in cs)


@pytest.mark.parametrize("recipe", [MX, NV])
def test_two_streams_at_once(recipe):
    streams, sides = [torch.cuda.Stream() for _ in range(2)], [calls(recipe), calls(recipe)]
    spaces = [torch.zeros(max(c.nbytes for c in cs), dtype=torch.uint8, device="cuda") for cs in sides]
    torch.cuda.synchronize()
    for i in range(100):
        for c0, c1 in zip(sides[0], reversed(sides[1])):
            assert c0(spaces[0], streams[0]) == 0 and c1(spaces[1], streams[1]) == 0
    torch.cuda.synchronize()
    assert gsa.grouped_gemm_status() == 0
    assert all(c.right() for cs in sides for c in cs)


def resident(region):
    """One flag a page of an anonymous mapping."""
    libc, n = ctypes.CDLL(None, use_errno=True), len(region) // mmap.PAGESIZE
    flags = (ctypes.c_ubyte * n)()
    at = ctypes.addressof(ctypes.c_char.from_buffer(region))
    assert libc.mincore(ctypes.c_void_p(at), ctypes.c_size_t(len(region)), flags) == 0
    return at, np.frombuffer(flags, np.uint8) & 1


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("side", ["a", "b"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_nothing_behind_an_operand_is_touched(recipe, side, shape):
    """One operand's codes in host memory that the GPU reads through the host's page tables, in a mapping of which only
    the pages with codes are populated: what the GPU reads becomes resident."""
    cuda, value = ctypes.CDLL("libcuda.so.1"), ctypes.c_int()
    for attribute in (88, 100):   # pageable memory access, by the host's page tables
        if cuda.cuDeviceGetAttribute(ctypes.byref(value), attribute, torch.cuda.current_device()) or not value.value:
            pytest.skip("the GPU does not read pageable host memory")
    c = Call(np.random.default_rng(41), *SHAPES[shape], recipe)
    codes = getattr(c, side).data[:-1]
    for first in (0, mmap.PAGESIZE - 4096):   # the operand's start within a page
        region = mmap.mmap(-1, 8 << 20, flags=mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS)
        region.madvise(mmap.MADV_NOHUGEPAGE)
        origin = 2 << 20
        region[origin + first:origin + first + codes.size] = codes.tobytes()
        at, before = resident(region)

        class Host:   # stands in for the tensor
            def data_ptr(self):
                return at + origin + first

            def numel(self):
                return codes.size

        (c.qa if side == "a" else c.qb)["col_data"] = Host()
        c.dw.fill_(float("nan"))
        ws = torch.empty(c.nbytes, dtype=torch.uint8, device="cuda")
        assert c(ws, torch.cuda.current_stream()) == 0
        torch.cuda.synchronize()
        touched = np.flatnonzero(resident(region)[1] & ~before)
        assert touched.size == 0, touched * mmap.PAGESIZE - origin - first - codes.size
        assert c.right()
