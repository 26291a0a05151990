"""The gated products with all the experts that they take: most of them without rows, rows for the last one only, one row each.
Refused: one more, and scales that are not in the tiled layout."""
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, dev_split
from test_gpu_grouped_glu import U, Case, forward_ref, gradient_ref, gsa_params, near

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

E = 256
SOME = [0] * E
for _e, _rows in ((0, 1), (1, 130), (7, 3), (128, 40), (254, 1), (255, 17)):
    SOME[_e] = _rows


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split", [SOME, [0] * (E - 1) + [5], [1] * E], ids=["some", "last", "one each"])
def test_all_experts(recipe, split):
    act = "clamped_swiglu"
    c = Case(90 + sum(split), recipe, split, 40, 192, 2, tail=9)
    more = {"act": act, "probs": c.probs, "params": gsa_params(act), "b_groups": 2, "out_dtype": torch.float32}
    near(gsa.grouped_glu(*c.args(), **more), *forward_ref(c, act), U)
    dx, bx, dp, bp = gradient_ref(c, act)
    got = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more)
    near(got[0], dx, bx, U)
    near(got[1], dp, bp, U)
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_refusals(recipe):
    c = Case(91, recipe, [3, 5], 128, 128, 1)
    a, b, split, m, n, k, _ = c.args()
    x = torch.zeros((m, k), device="cuda")
    many = {key: torch.zeros(v.numel() * 129, dtype=v.dtype, device="cuda") for key, v in b.items()}
    rows = dict(a, amax_row=torch.ones(257, device="cuda"))
    for call in (lambda q, s: gsa.grouped_glu(rows, q, s, m, n, k, recipe), lambda q, s: gsa.grouped_glu_bwd(c.dy_dev, rows, q, s, m, n, k, recipe),
                 lambda q, s: gsa.grouped_gemv(x, q, s, n, recipe), lambda q, s: gsa.grouped_glu_gemv(x, q, s, n, recipe)):
        with pytest.raises(gsa.GsaError):
            call(many, dev_split([0] * 257))
        compact = dict(b, row_scale=b["row_scale"].clone())
        gsa._record_layout(compact, gsa.SCALES_COMPACT, ("row_scale",))
        with pytest.raises(gsa.GsaError, match="compact"):
            call(compact, split)
