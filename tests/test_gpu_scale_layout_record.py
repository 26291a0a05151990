"""What fwd and bwd write, host split or device split, is refused by the products where its scales are compact."""
import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("recipe", [gsa.MXFP8, gsa.NVFP4])
@pytest.mark.parametrize("graph_safe", [False, True])
def test_written_copies(recipe, graph_safe):
    split, m, w = [128, 256], 384, 512
    s = torch.tensor(split, device="cuda")
    fwd, bwd = (gsa.fwd_graph_safe, gsa.bwd_graph_safe) if graph_safe else (gsa.fwd, gsa.bwd)
    given = s if graph_safe else split
    x = torch.ones((m, w), dtype=torch.bfloat16, device="cuda")

    def product(q):
        return gsa.grouped_gemm(q, q, s, m, 128, w, recipe)

    def wgrad(q):
        return gsa.grouped_gemm_wgrad(q, q, s, m, w, w, recipe)

    tiled = fwd(x, None, given, "identity", recipe, scale_layout=gsa.SCALES_TILED)
    grad = bwd(x, x, None, given, "srelu", recipe, regen=True, scale_layout=gsa.SCALES_TILED)
    again = {k[2:]: v for k, v in grad.items() if k.startswith("y_")}
    for q in (tiled, grad, again):
        wgrad(q)
    product(tiled), product(grad)
    assert gsa.grouped_gemm_status() == 0
    compact = fwd(x, None, given, "identity", recipe)
    grad = bwd(x, x, None, given, "srelu", recipe, regen=True)
    again = {k[2:]: v for k, v in grad.items() if k.startswith("y_")}
    for call in [lambda q=q: product(q) for q in (compact, grad)] + [lambda q=q: wgrad(q) for q in (compact, grad, again)]:
        with pytest.raises(gsa.GsaError, match="compact"):
            call()
    fwd(x, None, given, "identity", recipe, out=tiled)   # the same buffers, written compact
    with pytest.raises(gsa.GsaError, match="compact"):
        product(tiled)
