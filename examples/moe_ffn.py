"""A mixture-of-experts FFN on quantized operands, forward and backward, from this library's calls alone.

    python examples/moe_ffn.py [--recipe mxfp8|nvfp4] [--tokens 4096] [--experts 16] [--topk 4] [--hidden 1024]
                               [--width 1024] [--act srelu]

Forward:  sort the routed tokens by expert -> gather their rows -> quantize -> first projection -> scaled activation
fused with the quantization of its result -> second projection -> sum each token's expert rows.
Backward: the same way back, with both input gradients, both weight gradients and the router probabilities' gradient.
The split stays on the device throughout: nothing waits for the host, and a step can be captured in a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_quantization_grouped_gb300 import gsa  # noqa: E402

T = gsa.SCALES_TILED


class MoeFfn:
    """Expert weights w1 [E, W_in, H] and w2 [E, H, W] (BF16; W_in = 2 W for the GLU activations), quantized once.

    NVFP4 takes the random Hadamard transform on the columnwise copies of activations and gradients (they meet only
    in weight gradients, where it cancels) and none on the weights' (they meet untransformed rows)."""

    def __init__(self, w1, w2, act="srelu", recipe=gsa.MXFP8, rht_mask=0xBEEF):
        self.experts, self.w_in, self.hidden = w1.shape
        self.width = w2.shape[2]
        self.act, self.recipe, self.rht, self.mask = act, recipe, recipe == gsa.NVFP4, rht_mask
        self.w1, self.w2 = self._weights(w1), self._weights(w2)

    def _weights(self, w):
        e, n, k = w.shape
        return gsa.fwd(w.reshape(e * n, k), None, [n] * e, "identity", self.recipe, scale_layout=T)

    def _quantize(self, rows, split):
        return gsa.fwd_graph_safe(rows, None, split, "identity", self.recipe, self.rht, self.mask, scale_layout=T)

    def forward(self, x, expert_idx, probs):
        """x [tokens, H] BF16, expert_idx [tokens, topk] (outside [0, E): dropped), probs [tokens, topk] FP32
        -> out [tokens, H] and what the backward needs."""
        r, e = self.recipe, self.experts
        row, split = gsa.moe_sort(expert_idx, e)
        split = gsa.moe_groups(split)                        # the dropped rows are the last group (or the last expert's)
        xs, ps = gsa.moe_permute(x, row, probs)
        m, used = xs.shape[0], split[:e]
        qx = self._quantize(xs, split)
        h = gsa.grouped_gemm(qx, self.w1, used, m, self.w_in, self.hidden, r)
        qy = gsa.fwd_graph_safe(h, ps, split, self.act, r, self.rht, self.mask, scale_layout=T)
        ys = gsa.grouped_gemm(qy, self.w2, used, m, self.hidden, self.width, r)
        return gsa.moe_unpermute(ys, row), (row, split, ps, qx, h, qy)   # the activation applied the probabilities

    def backward(self, dout, saved):
        """-> dx [tokens, H] BF16, dprobs [tokens, topk] FP32, dw1 and dw2 FP32."""
        row, split, ps, qx, h, qy = saved
        r, e = self.recipe, self.experts
        m, used = h.shape[0], split[:e]
        dys, _ = gsa.moe_unpermute_bwd(dout, None, row)
        qd = self._quantize(dys, split)
        dy = gsa.grouped_gemm(qd, self.w2, used, m, self.width, self.hidden, r, b_columnwise=True)
        dw2 = gsa.grouped_gemm_wgrad(qd, qy, used, m, self.hidden, self.width, r)
        g = gsa.bwd_graph_safe(dy, h, ps, split, self.act, r, self.rht, self.mask, scale_layout=T)
        dxs = gsa.grouped_gemm(g, self.w1, used, m, self.hidden, self.w_in, r, b_columnwise=True)
        dw1 = gsa.grouped_gemm_wgrad(g, qx, used, m, self.w_in, self.hidden, r)
        dx, dprobs = gsa.moe_permute_bwd(dxs, row, g["dprobs"])
        return dx, dprobs, dw1, dw2


def reference(x, idx, probs, w1, w2, dout, act):
    """The same step in FP32 autograd on unquantized operands, expert by expert (srelu or identity)."""
    x, probs, w1, w2 = (t.float().requires_grad_() for t in (x, probs, w1, w2))
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if tok.numel():
            h = x[tok] @ w1[e].t()
            a = torch.relu(h) ** 2 if act == "srelu" else h
            out = out.index_add(0, tok, (probs[tok, slot][:, None] * a) @ w2[e].t())
    out.backward(dout.float())
    return out.detach(), x.grad, probs.grad, w1.grad, w2.grad


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--recipe", choices=("mxfp8", "nvfp4"), default="mxfp8")
    ap.add_argument("--act", default="srelu", choices=("srelu", "identity"))
    for name, value in (("tokens", 4096), ("experts", 16), ("topk", 4), ("hidden", 1024), ("width", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    w1 = normal(a.experts, a.width, a.hidden, scale=a.hidden ** -0.5)
    w2 = normal(a.experts, a.hidden, a.width, scale=a.width ** -0.5)
    x, dout = normal(a.tokens, a.hidden), normal(a.tokens, a.hidden)
    logits = torch.randn((a.tokens, a.experts), generator=g, device="cuda")
    probs, idx = torch.topk(torch.softmax(logits, 1), a.topk)
    ffn = MoeFfn(w1, w2, a.act, gsa.MXFP8 if a.recipe == "mxfp8" else gsa.NVFP4)

    def step():
        out, saved = ffn.forward(x, idx, probs)
        return (out, *ffn.backward(dout, saved))

    got = step()
    assert gsa.grouped_gemm_status() == 0
    for name, u, v in zip(("out", "dx", "dprobs", "dw1", "dw2"), got, reference(x, idx, probs, w1, w2, dout, a.act)):
        print("%-7s relative error against FP32 on unquantized operands: %.3f" % (name, float((u.float() - v).norm() / v.norm())))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        step()
    start.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    print("forward + backward: %.1f us" % (start.elapsed_time(end) * 100))


if __name__ == "__main__":
    main()
