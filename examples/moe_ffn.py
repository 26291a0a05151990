"""A mixture-of-experts FFN on quantized operands, forward and backward, from this library's calls alone.

    python examples/moe_ffn.py [--recipe mxfp8|nvfp4] [--tokens 4096] [--experts 16] [--topk 4] [--hidden 1024]
                               [--width 1024] [--act srelu|identity|swiglu]

Forward:  sort the routed tokens by expert -> gather their rows -> quantize -> first projection -> scaled activation
fused with the quantization of its result -> second projection -> sum each token's expert rows.
Backward: the same way back, with both input gradients, both weight gradients and the router probabilities' gradient.
Gated activations of widths that are multiples of 128 can be the first projection's epilogue: its result is then not written
in front of the activation, and the backward multiplies again instead of keeping it.  NVFP4 steps and forwards that no
backward follows do so; MXFP8 steps, in which the second multiplication costs more than the writing, are made of the
separate calls unless the memory matters more (recompute=True).
Decoding: both projections of a few rows an expert without quantizing them (gated activations).
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
    in weight gradients, where it cancels) and none on the weights' (they meet untransformed rows).

    recompute: whether the step of a gated FFN keeps no pre-activations (4 W bytes a row less) and multiplies again in the
    backward.  None: where that is faster.  Steps in a graph with and without, ms, 8192 tokens to 8 of 32 experts, H and W
    2048, and 32768 to 8 of 128, W 4096: NVFP4 2.59 / 2.71 and 16.7 / 17.9, MXFP8 2.96 to 3.02 / 2.87 to 2.89 and 22.7 to
    23.2 / 21.1 to 21.3 (4096 tokens to 4 of 16, H and W 1024: 0.45 / 0.47 and 0.415 / 0.42)."""

    def __init__(self, w1, w2, act="srelu", recipe=gsa.MXFP8, rht_mask=0xBEEF, recompute=None):
        self.experts, self.w_in, self.hidden = w1.shape
        self.width = w2.shape[2]
        self.act, self.recipe, self.rht, self.mask = act, recipe, recipe == gsa.NVFP4, rht_mask
        self.gated = act in ("swiglu", "clamped_swiglu")
        self.fused = self.gated and self.width % 128 == 0   # the activation may be the first projection's epilogue
        self.recompute = recipe == gsa.NVFP4 if recompute is None else recompute
        self.w1, self.w2 = self._weights(w1), self._weights(w2)
        self.w1_sides = self._by_side(self.w1) if self.gated and not self.fused else None

    def _weights(self, w):
        e, n, k = w.shape
        return gsa.fwd(w.reshape(e * n, k), None, [n] * e, "identity", self.recipe, scale_layout=T)

    def _by_side(self, q):
        """The rowwise copy of w1 as gate rows and linear rows of their own (b_groups = 2), for widths that are no multiple of
        128: the same codes, block scales and units; the linear rows' scales start on a tile."""
        e, w = self.experts, self.width
        before, after = -(-2 * w // 128), -(-w // 128)
        c4 = q["row_scale"].numel() // (e * before * 512)
        rows = q["row_scale"].view(e, before, c4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(e, before * 128, 4 * c4)
        scale = rows.new_zeros((2 * e, after * 128, 4 * c4))
        scale[:, :w] = rows[:, :2 * w].reshape(2 * e, w, 4 * c4)
        sides = {"row_data": q["row_data"], "row_scale": scale.view(2 * e, after, 4, 32, c4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)}
        if self.recipe == gsa.NVFP4:
            sides["amax_row"] = q["amax_row"].repeat_interleave(2)
        return sides

    def _quantize(self, rows, split):
        return gsa.fwd_graph_safe(rows, None, split, "identity", self.recipe, self.rht, self.mask, scale_layout=T)

    def forward(self, x, expert_idx, probs, train=True):
        """x [tokens, H] BF16, expert_idx [tokens, topk] (outside [0, E): dropped), probs [tokens, topk] FP32
        -> out [tokens, H] and what the backward needs.  train=False: no backward follows, whose needs then do not decide
        how the activation is made (a backward that does follow multiplies again)."""
        r, e = self.recipe, self.experts
        row, split = gsa.moe_sort(expert_idx, e)
        split = gsa.moe_groups(split)                        # the dropped rows are the last group (or the last expert's)
        xs, ps = gsa.moe_permute(x, row, probs)
        m, used = xs.shape[0], split[:e]
        qx = self._quantize(xs, split)
        if self.fused and (self.recompute or not train):
            h = None
            qy = self._quantize(gsa.grouped_glu(qx, self.w1, used, m, self.width, self.hidden, r, self.act, ps), split)
        else:
            h = gsa.grouped_gemm(qx, self.w1, used, m, self.w_in, self.hidden, r)
            qy = gsa.fwd_graph_safe(h, ps, split, self.act, r, self.rht, self.mask, scale_layout=T)
        ys = gsa.grouped_gemm(qy, self.w2, used, m, self.hidden, self.width, r)
        return gsa.moe_unpermute(ys, row), (row, split, ps, qx, h, qy)   # the activation applied the probabilities

    def backward(self, dout, saved):
        """-> dx [tokens, H] BF16, dprobs [tokens, topk] FP32, dw1 and dw2 FP32."""
        row, split, ps, qx, h, qy = saved
        r, e = self.recipe, self.experts
        m, used = ps.shape[0], split[:e]
        dys, _ = gsa.moe_unpermute_bwd(dout, None, row)
        qd = self._quantize(dys, split)
        dy = gsa.grouped_gemm(qd, self.w2, used, m, self.width, self.hidden, r, b_columnwise=True)
        dw2 = gsa.grouped_gemm_wgrad(qd, qy, used, m, self.hidden, self.width, r)
        if h is None:
            dh, dps = gsa.grouped_glu_bwd(dy, qx, self.w1, used, m, self.width, self.hidden, r, self.act, ps)
            g = dict(self._quantize(dh, split), dprobs=dps)
        else:
            g = gsa.bwd_graph_safe(dy, h, ps, split, self.act, r, self.rht, self.mask, scale_layout=T)
        dxs = gsa.grouped_gemm(g, self.w1, used, m, self.hidden, self.w_in, r, b_columnwise=True)
        dw1 = gsa.grouped_gemm_wgrad(g, qx, used, m, self.w_in, self.hidden, r)
        dx, dprobs = gsa.moe_permute_bwd(dxs, row, g["dprobs"])
        return dx, dprobs, dw1, dw2

    def decode(self, x, expert_idx, probs):
        """The forward of a few tokens [tokens, H] (BF16, FP16 or FP32), rows as they are against the quantized weights."""
        row, split = gsa.moe_sort(expert_idx, self.experts)
        xs, ps = gsa.moe_permute(x, row, probs)
        used = split[:self.experts]
        w1, groups = (self.w1, 1) if self.fused else (self.w1_sides, 2)
        y = gsa.grouped_glu_gemv(xs, w1, used, self.width, self.recipe, self.act, ps, b_groups=groups)
        return gsa.moe_unpermute(gsa.grouped_gemv(y, self.w2, used, self.hidden, self.recipe), row)


def reference(x, idx, probs, w1, w2, dout, act):
    """The same step in FP32 autograd on unquantized operands, expert by expert (srelu, identity or swiglu)."""
    x, probs, w1, w2 = (t.float().requires_grad_() for t in (x, probs, w1, w2))
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if tok.numel():
            h = x[tok] @ w1[e].t()
            gate, linear = h.chunk(2, 1)
            a = torch.relu(h) ** 2 if act == "srelu" else gate * torch.sigmoid(gate) * linear if act == "swiglu" else h
            out = out.index_add(0, tok, (probs[tok, slot][:, None] * a) @ w2[e].t())
    out.backward(dout.float())
    return out.detach(), x.grad, probs.grad, w1.grad, w2.grad


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--recipe", choices=("mxfp8", "nvfp4"), default="mxfp8")
    ap.add_argument("--act", default="srelu", choices=("srelu", "identity", "swiglu"))
    for name, value in (("tokens", 4096), ("experts", 16), ("topk", 4), ("hidden", 1024), ("width", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    w1 = normal(a.experts, a.width * (2 if a.act == "swiglu" else 1), a.hidden, scale=a.hidden ** -0.5)
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
    if ffn.gated:
        few = slice(0, 4)
        u, v = ffn.decode(x[few], idx[few].contiguous(), probs[few].contiguous()), got[0][few]
        print("decode  against the forward's rows: %.3f" % float((u.float() - v.float()).norm() / v.float().norm()))


if __name__ == "__main__":
    main()
