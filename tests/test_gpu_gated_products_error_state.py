"""An error that another call has left in the CUDA runtime is not taken for one of the gated products'.  The failure is the host's:
a stream whose capture has been invalidated (test_gpu_moe_error_state)."""
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV
from test_gpu_grouped_glu import Case
from test_gpu_moe_error_state import BrokenCapture, qin

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("recipe", [MX, NV])
def test_errors_of_other_calls(recipe):
    n, k = 256, 64
    c = Case(55, recipe, [30, 40], n, k, 1)
    L, shape, side = gsa.load(), (2, c.m, n, k, recipe), torch.cuda.Stream()
    a, b, sp = qin(c.qa, "row"), qin(c.qb, "row"), c.dev.data_ptr()
    y, dx, dp = torch.empty((c.m, n), device="cuda"), torch.empty((c.m, 2 * n), device="cuda"), torch.empty(c.m, device="cuda")
    x, out, gated = torch.randn((c.m, k), device="cuda"), torch.empty((c.m, n), device="cuda"), torch.empty((c.m, n), device="cuda")
    n_bwd, n_few = L.gsa_grouped_glu_bwd_workspace_size(c.m, n), L.gsa_grouped_gemv_workspace_size(2, c.m, k, recipe)
    ws = torch.empty(max(n_bwd, n_few), dtype=torch.uint8, device="cuda")
    header = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    want = (gsa.grouped_glu(*c.args(), out_dtype=torch.float32), *gsa.grouped_glu_bwd(c.dy_dev, *c.args(), out_dtype=torch.float32),
            gsa.grouped_gemv(x, c.qb, c.dev, n, recipe), gsa.grouped_glu_gemv(x, c.qb, c.dev, n, recipe))
    torch.cuda.synchronize()
    calls = (lambda s: L.gsa_grouped_glu(a, b, sp, *shape, 2, None, None, 1, y.data_ptr(), gsa.FP32, s),
             lambda s: L.gsa_grouped_glu_bwd(c.dy_dev.data_ptr(), a, b, sp, *shape, 2, None, None, 1, dx.data_ptr(), gsa.FP32, dp.data_ptr(),
                                             ws.data_ptr(), n_bwd, s),
             lambda s: L.gsa_grouped_gemv(x.data_ptr(), gsa.FP32, b, sp, *shape, out.data_ptr(), gsa.FP32, ws.data_ptr(), n_few, s),
             lambda s: L.gsa_grouped_glu_gemv(x.data_ptr(), gsa.FP32, b, sp, *shape, 2, None, None, 1, gated.data_ptr(), gsa.FP32, ws.data_ptr(), n_few, s))
    row, t, ts = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), torch.ones((4, 64), device="cuda"), torch.empty((8, 64), device="cuda")
    got = []
    with BrokenCapture() as stream:
        for call in calls:
            assert L.gsa_selftest_wait_timeout(header.data_ptr(), 0, 1, stream) == 5   # fails before any launch
            got.append(call(side.cuda_stream))
    # takes the error out of the runtime, that no other test meets it
    L.gsa_moe_permute(t.data_ptr(), None, row.data_ptr(), 4, 2, 64, gsa.FP32, ts.data_ptr(), None, side.cuda_stream)
    torch.cuda.synchronize()
    assert got == [0, 0, 0, 0]
    assert all(torch.equal(u, v) for u, v in zip((y, dx, dp, out, gated), want)) and gsa.grouped_gemm_status() == 0
