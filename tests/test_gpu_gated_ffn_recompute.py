"""Gated steps with the pre-activations kept and with them multiplied again: which of them runs, that both are the step's
gradients, and that a forward without a backward takes the fused projection."""
import pytest
import torch

from test_gpu_gated_ffn import problem
from test_gpu_grouped_gemm import MX, NV
from test_gpu_moe_chain import example

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


class Counted:
    """How often the fused projection, its gradient and the separate activation run."""

    def __init__(self, monkeypatch):
        self.calls = []
        for name in ("grouped_glu", "grouped_glu_bwd", "bwd_graph_safe"):
            monkeypatch.setattr(gsa, name, self.of(name, getattr(gsa, name)))

    def of(self, name, f):
        def call(*args, **more):
            self.calls.append(name)
            return f(*args, **more)
        return call


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("recompute", [None, False, True])
@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
def test_step(monkeypatch, recipe, recompute, act):
    """Both steps have the same operands but for pre-activations rounded to BF16 or not, which moves y and its gradients by
    d = 2 2^-8 at most.  A value that moves by d before it is rounded to codes of relative step h goes to the neighbour
    with probability d / h: sqrt(d h) in the norm, 2^-5 for E4M3 (h = 2^-3), 2^-4 for E2M1 (2^-1); each result has one such
    operand.  Half of the codes' own error (2^-4; 2^-2 and the scales' 2^-4) covers that and the scales that change."""
    ex = example()
    w1, w2, x, dout, probs, idx = problem(21, 5, 700, 2, 192, 256)
    ffn = ex.MoeFfn(w1, w2, act, recipe, recompute=recompute)
    assert ffn.recompute == (recipe == NV if recompute is None else recompute)
    count = Counted(monkeypatch)
    out, saved = ffn.forward(x, idx, probs)
    got = (out, *ffn.backward(dout, saved))
    assert count.calls == (["grouped_glu", "grouped_glu_bwd"] if ffn.recompute else ["bwd_graph_safe"])
    del count.calls[:]
    ffn.recompute = not ffn.recompute
    out, saved = ffn.forward(x, idx, probs)
    other = (out, *ffn.backward(dout, saved))
    assert count.calls == (["grouped_glu", "grouped_glu_bwd"] if ffn.recompute else ["bwd_graph_safe"])
    assert gsa.grouped_gemm_status() == 0
    half = (2.0 ** -4 if recipe == MX else 2.0 ** -2 + 2.0 ** -4) / 2
    for name, u, v in zip(("out", "dx", "dprobs", "dw1", "dw2"), got, other):
        assert float((u.float() - v.float()).norm() / v.float().norm()) <= 2 * 2.0 ** -8 + half, name


@pytest.mark.parametrize("recipe", [MX, NV])
def test_forward_alone(monkeypatch, recipe):
    ex = example()
    w1, w2, x, dout, probs, idx = problem(22, 4, 300, 2, 128, 256)
    ffn = ex.MoeFfn(w1, w2, "swiglu", recipe, recompute=False)
    count = Counted(monkeypatch)
    out, saved = ffn.forward(x, idx, probs, train=False)
    assert count.calls == ["grouped_glu"]
    got = (out, *ffn.backward(dout, saved))   # it can follow all the same
    assert count.calls == ["grouped_glu", "grouped_glu_bwd"]
    ffn.recompute = True
    out, saved = ffn.forward(x, idx, probs)
    assert all(torch.equal(u, v) for u, v in zip(got, (out, *ffn.backward(dout, saved))))
    odd = ex.MoeFfn(w1[:, :384].contiguous(), w2[:, :, :192].contiguous(), "swiglu", recipe)
    del count.calls[:]
    odd.forward(x, idx, probs, train=False)
    assert count.calls == [] and gsa.grouped_gemm_status() == 0
