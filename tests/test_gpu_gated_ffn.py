"""The gated expert FFN from the library's calls together, as the example makes them: training step and decoding.

Against FP32 on unquantized operands: each quantized operand is within 2^-4 (E4M3) or 2^-2 (E2M1, plus 2^-4 of its scale) of
itself, and the errors of those that a result goes through are independent, so that they add in quadrature.  x and w1 enter
the output twice (gate and linear side), as the squared activation's do."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, decode_copy
from test_gpu_moe_chain import example

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def problem(seed, e, t, topk, hidden, width, drop=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    w1, w2 = normal(e, 2 * width, hidden, scale=hidden ** -0.5), normal(e, hidden, width, scale=width ** -0.5)
    x, dout = normal(t, hidden), normal(t, hidden)
    probs, idx = torch.topk(torch.softmax(torch.randn((t, e), generator=g, device="cuda"), 1), topk)
    if drop:
        idx[::7, 1] = -1
        idx[t // 2] = -1
    return w1, w2, x, dout, probs, idx


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("e,t,topk,hidden,width", [(6, 500, 2, 192, 256), (4, 2000, 2, 256, 128), (5, 300, 2, 128, 192)], ids=str)
def test_training_step(recipe, e, t, topk, hidden, width):
    """The last width is no multiple of 128: the example then makes the step of separate calls."""
    ex = example()
    w1, w2, x, dout, probs, idx = problem(3, e, t, topk, hidden, width)
    ffn = ex.MoeFfn(w1, w2, "swiglu", recipe)
    assert ffn.fused == (width % 128 == 0)
    out, saved = ffn.forward(x, idx, probs)
    got = (out, *ffn.backward(dout, saved))
    assert gsa.grouped_gemm_status() == 0
    one = 2.0 ** -4 if recipe == MX else 2.0 ** -2 + 2.0 ** -4
    for name, u, v, operands in zip(("out", "dx", "dprobs", "dw1", "dw2"), got, ex.reference(x, idx, probs, w1, w2, dout, "swiglu"),
                                    (6, 8, 6, 8, 6)):
        err = float((u.float() - v).norm() / v.norm())
        assert err <= operands ** 0.5 * one, (name, err)
        # the projection on the reference shows a lost factor or term: rounded operands q = x + d have <d, x> about -|d|^2
        along = float((u.float() * v).sum() / (v * v).sum())
        assert abs(along - 1) <= operands * (one / 3) ** 2 + 0.05, (name, along)
    dropped = idx[t // 2] < 0
    assert bool(dropped.all()) and bool((got[0][t // 2] == 0).all()) and bool((got[1][t // 2] == 0).all()) and bool((got[2][idx < 0] == 0).all())


@pytest.mark.parametrize("recipe", [MX, NV])
def test_step_in_a_graph(recipe):
    """Forward, backward and a decoding step captured together and replayed with other tokens and another routing in place:
    the bits of the eager calls."""
    ex = example()
    a, b = (problem(s, 6, 200, 2, 192, 256) for s in (5, 6))
    ffn = ex.MoeFfn(a[0], a[1], "swiglu", recipe)
    x, dout, probs, idx = (v.clone() for v in a[2:])

    def step():
        out, saved = ffn.forward(x, idx, probs)
        return (out, *ffn.backward(dout, saved), ffn.decode(x[:8], idx[:8], probs[:8]))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for p in (b, a):
        for to, v in zip((x, dout, probs, idx), p[2:]):
            to.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(u, v) for u, v in zip(outs, want))
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("tokens,topk,e,hidden,width", [(1, 2, 4, 128, 128), (1, 8, 128, 256, 256), (7, 3, 5, 320, 384), (64, 2, 8, 192, 128)], ids=str)
def test_decoding(recipe, tokens, topk, e, hidden, width):
    """Against FP64 with the decoded weights.  y is rounded to BF16 (2^-8), which the second product turns into 2^-8 of its
    sum of magnitudes; so is each of its results, and the sum over a token's experts: 3 times 2^-8 of the magnitudes at most,
    and FP32's errors (2^-16 of them, and of the activation's arguments, is generous)."""
    ex = example()
    w1, w2, x, _, probs, idx = problem(7, e, tokens, topk, hidden, width, drop=tokens > 2)
    ffn = ex.MoeFfn(w1, w2, "swiglu", recipe)
    got = ffn.decode(x, idx, probs).double().cpu().numpy()
    assert gsa.grouped_gemm_status() == 0
    d1 = decode_copy(ffn.w1, "row", recipe, [2 * width] * e, hidden)
    d2 = decode_copy(ffn.w2, "row", recipe, [hidden] * e, width)
    ref, mass = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    xs, ps, ix = x.double().cpu().numpy(), probs.double().cpu().numpy(), idx.cpu().numpy()
    for t in range(tokens):
        for j in range(topk):
            if ix[t, j] < 0:
                continue
            h = d1[ix[t, j]] @ xs[t]
            y = ps[t, j] * h[:width] / (1 + np.exp(-h[:width])) * h[width:]
            ref[t] += d2[ix[t, j]] @ y
            mass[t] += np.abs(d2[ix[t, j]]) @ np.abs(y)
    assert np.all(np.abs(got - ref) <= (3 * 2.0 ** -8 + 2.0 ** -16) * mass + 2.0 ** -16)


def test_decoding_agrees_with_the_forward():
    """The same tokens through both forms: they differ by the quantization of the rows alone."""
    ex = example()
    w1, w2, x, _, probs, idx = problem(9, 8, 64, 2, 256, 256, drop=False)
    for recipe, one in ((MX, 2.0 ** -4), (NV, 2.0 ** -2 + 2.0 ** -4)):
        ffn = ex.MoeFfn(w1, w2, "swiglu", recipe)
        u, v = ffn.decode(x, idx, probs).float(), ffn.forward(x, idx, probs)[0].float()
        assert float((u - v).norm() / v.norm()) <= 3 ** 0.5 * one   # x twice, y once
