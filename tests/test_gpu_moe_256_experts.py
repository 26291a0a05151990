"""The whole mixture-of-experts step with as many experts as the operators take, and dropped slots: 200 experts numbered
56 .. 255 give bit for bit what the same 200 give numbered 0 .. 199."""
import importlib.util
import os

import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_ffn.py")
    spec = importlib.util.spec_from_file_location("moe_ffn", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


@pytest.mark.parametrize("recipe", [gsa.MXFP8, gsa.NVFP4])
@pytest.mark.parametrize("drop", [0.0, 0.2, 1.0])
def test_step_with_256_experts(recipe, drop):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    tokens, topk, hidden, width, few, many = 700, 3, 128, 64, 200, 256

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    w1, w2 = normal(many, width, hidden), normal(many, hidden, width)
    x, dout = normal(tokens, hidden), normal(tokens, hidden)
    idx = torch.rand((tokens, few), generator=g, device="cuda").topk(topk).indices
    gone = torch.rand((tokens, topk), generator=g, device="cuda") < drop
    probs = torch.rand((tokens, topk), generator=g, device="cuda")
    ffn = example().MoeFfn
    results = []
    for shift, experts in ((0, few), (many - few, many)):
        step = ffn(w1[many - few:] if shift == 0 else w1, w2[many - few:] if shift == 0 else w2, "srelu", recipe)
        out, saved = step.forward(x, torch.where(gone, -1, idx + shift), probs)
        results.append((out, *step.backward(dout, saved)))
        assert gsa.grouped_gemm_status() == 0
    for name, u, v in zip(("out", "dx", "dprobs"), results[0], results[1]):
        assert torch.equal(u, v), name
    for name, u, v in zip(("dw1", "dw2"), results[0][3:], results[1][3:]):
        assert torch.equal(u, v[many - few:]) and bool((v[:many - few] == 0).all()), name


def test_groups():
    split = torch.arange(13, device="cuda")
    assert gsa.moe_groups(split) is split
    split = torch.arange(257, device="cuda")
    groups = gsa.moe_groups(split)
    assert groups.cpu().tolist() == list(range(255)) + [255 + 256] and split.cpu().tolist() == list(range(257))
