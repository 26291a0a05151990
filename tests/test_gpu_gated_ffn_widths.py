"""Decoding through gated experts whose width is no multiple of 128: the linear rows' scales then start inside a tile of w1, and
the example lays them out anew.  Bounds as in test_gpu_gated_ffn."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_gated_ffn import problem
from test_gpu_grouped_gemm import MX, NV, decode_copy
from test_gpu_moe_chain import example

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("tokens,topk,e,hidden,width", [(1, 2, 4, 128, 192), (7, 3, 5, 320, 64), (30, 2, 3, 192, 448), (9, 8, 200, 64, 64)], ids=str)
def test_decoding(recipe, tokens, topk, e, hidden, width):
    ex = example()
    w1, w2, x, _, probs, idx = problem(11, e, tokens, topk, hidden, width, drop=tokens > 2)
    ffn = ex.MoeFfn(w1, w2, "swiglu", recipe)
    assert not ffn.fused
    got = ffn.decode(x, idx, probs).double().cpu().numpy()
    assert gsa.grouped_gemm_status() == 0
    d1 = decode_copy(ffn.w1, "row", recipe, [2 * width] * e, hidden)
    sides = decode_copy(ffn.w1_sides, "row", recipe, [width] * (2 * e), hidden)
    d2 = decode_copy(ffn.w2, "row", recipe, [hidden] * e, width)
    assert all(np.array_equal(v, np.concatenate(sides[2 * i:2 * i + 2])) for i, v in enumerate(d1))
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


@pytest.mark.parametrize("recipe", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("width", [192, 256])
def test_the_command(recipe, width):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cmd = [sys.executable, os.path.join(root, "examples", "moe_ffn.py"), "--recipe", recipe, "--act", "swiglu", "--tokens", "300", "--experts", "5",
           "--topk", "2", "--hidden", "128", "--width", str(width)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "decode" in r.stdout, r.stdout + r.stderr
