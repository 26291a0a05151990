"""A call that fails in the CUDA runtime leaves no error behind for the next one.  The failure is the host's: a stream whose
capture has been invalidated."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split, padded

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


class BrokenCapture:
    """A stream in a capture that a forbidden call ended; its launches fail."""

    def __enter__(self):
        self.cuda, self.stream = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
        assert self.cuda.cuStreamCreate(ctypes.byref(self.stream), 1) == 0
        assert self.cuda.cuStreamBeginCapture_v2(self.stream, 1) == 0   # thread-local
        assert self.cuda.cuStreamSynchronize(self.stream) != 0
        return self.stream

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        assert self.cuda.cuStreamEndCapture(self.stream, ctypes.byref(graph)) != 0
        assert self.cuda.cuStreamDestroy_v2(self.stream) == 0


def qin(q, side):
    return gsa.QIn(q[side + "_data"].data_ptr(), q[side + "_scale"].data_ptr(), q["amax_" + side].data_ptr(),
                   q[side + "_data"].numel(), q[side + "_scale"].numel())


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("rows", [10, 400])   # single blocks, pairs
def test_failed_launch_leaves_no_error(recipe, rows):
    rng = np.random.default_rng(51)
    split, n, k = [rows, rows], 160, 192
    mp = padded(split, recipe)
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * 2, k, recipe)
    qa, qb, s = a.dev(), b.dev(), dev_split(split)
    ca, cb = Matrices(rng, [n] * 2, mp, recipe).dev("col"), Matrices(rng, [k] * 2, mp, recipe).dev("col")
    out, dw = torch.empty((2 * rows, n), device="cuda"), torch.empty((2, n, k), device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    row, x = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), torch.ones((4, 64), device="cuda")
    xs = torch.empty((8, 64), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    L, shape = gsa.load(), (2, 2 * rows, n, k, recipe)
    with BrokenCapture() as stream:
        for call in (lambda: L.gsa_grouped_gemm(qin(qa, "row"), qin(qb, "row"), s.data_ptr(), *shape, out.data_ptr(), gsa.FP32, stream),
                     lambda: L.gsa_grouped_gemm_wgrad(qin(ca, "col"), qin(cb, "col"), s.data_ptr(), *shape, dw.data_ptr(), gsa.FP32, 0,
                                                      ws.data_ptr(), ws.numel(), stream),
                     lambda: L.gsa_grouped_gemm_status(stream)):
            assert call() == 5
            # a good call on another stream, which looks at the error state behind its launch
            assert L.gsa_moe_permute(x.data_ptr(), None, row.data_ptr(), 4, 2, 64, gsa.FP32, xs.data_ptr(), None,
                                     side.cuda_stream) == 0
    torch.cuda.synchronize()
    got = gsa.grouped_gemm(qa, qb, s, 2 * rows, n, k, recipe, out_dtype=torch.float32)
    assert gsa.grouped_gemm_status() == 0 and bool((xs == 1).all())
    assert np.array_equal(got.double().cpu().numpy(), np.concatenate([u @ w.T for u, w in zip(a.values, b.values)]))
