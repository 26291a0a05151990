"""The whole mixture-of-experts step, call by call and end to end.

Every grouped product that the step makes is compared with the FP64 product of the decoded copies that it was given: off
by at most K 2^-23 of the sum of magnitudes, and 2^-8 (BF16) or 2^-22 (FP32) of the result for its own rounding.

End to end, against FP32 on unquantized operands, a lost factor or term has to show.  An operand that is rounded to
nearest is q = x + d with <d, x> about -|d|^2, and the errors of different operands are independent.  With e_i the
measured |d| / |x| of each operand and m_i how often it enters (the squared activation doubles what is inside), the
relative error is about sqrt(sum m_i^2 e_i^2), taken 1.5 times, and the projection <got, ref> / <ref, ref> is 1 within
sum m_i e_i^2 + 0.05.  Half a result, or one of a token's two experts missing, is off by 0.3 and more."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, decode_copy, dev_split, padded

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


def near(got, pairs, terms, rel):
    ref = np.concatenate([a @ b.T for a, b in pairs])
    mass = np.concatenate([np.abs(a) @ np.abs(b).T for a, b in pairs])
    got = got.double().cpu().numpy().reshape(-1, ref.shape[1])
    assert np.all(np.abs(got[:len(ref)] - ref) <= terms * 2.0 ** -23 * mass + rel * np.abs(ref))
    return got[len(ref):]


class Checked:
    """Stands in for grouped_gemm and grouped_gemm_wgrad: makes the call, then compares it."""

    def __init__(self, monkeypatch, groups):
        self.groups, self.made = groups, []
        self.gemm, self.wgrad = gsa.grouped_gemm, gsa.grouped_gemm_wgrad
        monkeypatch.setattr(gsa, "grouped_gemm", self.checked_gemm)
        monkeypatch.setattr(gsa, "grouped_gemm_wgrad", self.checked_wgrad)

    def checked_gemm(self, a, b, split, m, n, k, recipe, out_dtype=None, b_columnwise=False):
        out = self.gemm(a, b, split, m, n, k, recipe, out_dtype, b_columnwise)
        e = split.shape[0]
        x = decode_copy(a, "row", recipe, self.groups, k)[:e]
        w = decode_copy(b, "col" if b_columnwise else "row", recipe, [n] * e, k)
        rest = near(out, list(zip(x, w)), k, 2.0 ** -8 if out.dtype is torch.bfloat16 else 2.0 ** -22)
        assert np.all(rest == 0)   # rows that no expert has
        self.made.append("input gradient" if b_columnwise else "product")
        return out

    def checked_wgrad(self, a, b, split, m, n, k, recipe):
        out = self.wgrad(a, b, split, m, n, k, recipe)
        e, g = split.shape[0], len(self.groups)
        mp = padded(self.groups, recipe)
        x, w = decode_copy(a, "col", recipe, [n] * g, mp)[:e], decode_copy(b, "col", recipe, [k] * g, mp)[:e]
        near(out, list(zip(x, w)), max(mp), 2.0 ** -22)
        self.made.append("weight gradient")
        return out


def error(q, side, recipe, rows, k, source):
    """|q - x| / |x| of a quantized copy against its source."""
    v = np.concatenate(decode_copy(q, side, recipe, rows, k))
    x = source.double().cpu().numpy().reshape(v.shape)
    return float(np.linalg.norm(v - x) / np.linalg.norm(x))


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("e,t,topk,hidden,width", [(6, 500, 2, 192, 256), (3, 700, 2, 320, 192)])
def test_step(monkeypatch, recipe, e, t, topk, hidden, width):
    ex = example()
    g = torch.Generator(device="cuda")
    g.manual_seed(e)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    w1, w2 = normal(e, width, hidden, scale=hidden ** -0.5), normal(e, hidden, width, scale=width ** -0.5)
    x, dout = normal(t, hidden), normal(t, hidden)
    probs, idx = torch.topk(torch.softmax(torch.randn((t, e), generator=g, device="cuda"), 1), topk)
    idx[::7, 1] = -1    # dropped slots
    idx[3] = -1         # a token that no expert takes
    ffn = ex.MoeFfn(w1, w2, "srelu", recipe)
    groups = [int((idx == i).sum()) for i in range(e)] + [int((idx < 0).sum())]
    checked = Checked(monkeypatch, groups)
    out, saved = ffn.forward(x, idx, probs)
    got = (out, *ffn.backward(dout, saved))
    assert gsa.grouped_gemm_status() == 0
    assert sorted(checked.made) == ["input gradient"] * 2 + ["product"] * 2 + ["weight gradient"] * 2

    row, split, ps, qx, h, qy = saved
    y = (torch.relu(h.float()) ** 2 * ps[:, None]).to(torch.bfloat16)
    qd = gsa.fwd_graph_safe(dout, None, dev_split([t]), "identity", recipe, scale_layout=gsa.SCALES_TILED)
    xs = gsa.moe_permute(x, row)
    ex_, ey, ed = (error(q, "row", recipe, rows, s.shape[1], s) for q, rows, s in
                   ((qx, groups, xs), (qy, groups, y), (qd, [t], dout)))
    e1, e2 = (error(q, "row", recipe, [v.shape[1]] * e, v.shape[2], v.reshape(-1, v.shape[2])) for q, v in ((ffn.w1, w1), (ffn.w2, w2)))
    # how often each operand's error enters: (x, w1, y, w2, dout and the gradient's second quantization)
    times = {"out": (2, 2, 1, 1, 0), "dx": (1, 2, 0, 1, 2), "dprobs": (2, 2, 0, 1, 1), "dw1": (2, 1, 0, 1, 2), "dw2": (2, 2, 1, 0, 1)}
    for (name, m), u, v in zip(times.items(), got, ex.reference(x, idx, probs, w1, w2, dout, "srelu")):
        u, v = u.double(), v.double()
        sizes = list(zip(m, (ex_, e1, ey, e2, ed)))
        rel, proj = float((u - v).norm() / v.norm()), float((u * v).sum() / (v * v).sum())
        assert rel <= 1.5 * sum((i * s) ** 2 for i, s in sizes) ** 0.5, (name, rel)
        assert abs(proj - 1) <= sum(i * s * s for i, s in sizes) + 0.05, (name, proj)
    assert bool((got[0][3] == 0).all()) and bool((got[1][3] == 0).all()) and bool((got[2][idx < 0] == 0).all())


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", [([5, 0, 130], 64, 192), ([700, 3, 0, 129], 257, 256), ([0, 513, 255, 1, 1000, 31], 512, 320),
                                       ([64] * 30, 100, 128), ([2000], 300, 640)], ids=str)
def test_input_gradient(recipe, split, n, k):
    """Rows [m, k] times the columnwise copies of weights [k, n'] (n' the width padded to what the quantizer takes), few
    rows an expert and many."""
    rng = np.random.default_rng(n + k)
    e, m, wide = len(split), sum(split), -(-n // 64) * 64

    def bf16(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)

    qd = gsa.fwd(bf16(m, k), None, split, "identity", recipe, scale_layout=gsa.SCALES_TILED)
    qw = gsa.fwd(bf16(e * k, wide), None, [k] * e, "identity", recipe, scale_layout=gsa.SCALES_TILED)
    for dtype, rel in ((torch.float32, 2.0 ** -22), (torch.bfloat16, 2.0 ** -8)):
        dx = gsa.grouped_gemm(qd, qw, dev_split(split), m, wide, k, recipe, out_dtype=dtype, b_columnwise=True)
        near(dx, list(zip(decode_copy(qd, "row", recipe, split, k), decode_copy(qw, "col", recipe, [wide] * e, k))), k, rel)
    assert gsa.grouped_gemm_status() == 0
