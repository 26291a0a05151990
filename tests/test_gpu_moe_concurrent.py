"""Calls inside a capture before any outside of one, and products on two streams at once."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

FIRST = """
import sys
sys.path[:0] = [ROOT, TESTS]
import numpy as np, torch
from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split, padded
from nvfp4_quantization_grouped_gb300 import gsa
rng = np.random.default_rng(61)
calls = []
for recipe in (MX, NV):
    for rows in (10, 400):   # single blocks, pairs
        split, n, k = [rows, rows], 160, 192
        mp = padded(split, recipe)
        a, b = Matrices(rng, split, k, recipe).dev(), Matrices(rng, [n] * 2, k, recipe).dev()
        c, d = Matrices(rng, [n] * 2, mp, recipe).dev("col"), Matrices(rng, [k] * 2, mp, recipe).dev("col")
        s = dev_split(split)
        calls.append(lambda a=a, b=b, s=s, m=2 * rows, r=recipe: gsa.grouped_gemm(a, b, s, m, 160, 192, r))
        calls.append(lambda c=c, d=d, s=s, m=2 * rows, r=recipe: gsa.grouped_gemm_wgrad(c, d, s, m, 160, 192, r))
for tokens in (50, 1500, 9000):
    idx = torch.from_numpy(rng.integers(-1, 5, (tokens, 3))).cuda()
    for width in (64, 65):
        x, dx = torch.randn((tokens, width), device="cuda"), torch.randn((tokens * 3, width), device="cuda")
        def step(idx=idx, x=x, dx=dx):
            row, split = gsa.moe_sort(idx, 5)
            xs = gsa.moe_permute(x, row)
            return torch.cat([gsa.moe_unpermute(xs, row), gsa.moe_permute_bwd(dx, row), *gsa.moe_unpermute_bwd(x, None, row)[:1]])
        calls.append(step)
torch.cuda.synchronize()
graphs = []
for call in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    graphs.append((g, out))
for (g, out), call in zip(graphs, calls):
    out.fill_(float("nan"))
    g.replay()
    assert torch.equal(out, call())
assert gsa.grouped_gemm_status() == 0
print("same", len(calls))
"""


def test_first_calls_of_a_process_in_captures():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.replace("ROOT", repr(os.path.dirname(tests))).replace("TESTS", repr(tests))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same", "14"], r.stdout + r.stderr


@pytest.mark.parametrize("recipe", [MX, NV])
def test_products_on_two_streams(recipe):
    rng = np.random.default_rng(62)
    cases = []
    for split, n, k in (([40, 3, 0, 100], 200, 256), ([600, 300], 300, 1024), ([1] * 30, 64, 512)):
        a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * len(split), k, recipe)
        cases.append((a.dev(), b.dev(), dev_split(split), sum(split), n, k,
                      np.concatenate([x @ w.T for x, w in zip(a.values, b.values)])))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[torch.empty((c[3], c[4]), device="cuda") for c in cases] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(100):
        for i in range(len(cases)):
            for s, stream in enumerate(streams):
                at = i if s == 0 else len(cases) - 1 - i
                a, b, split, m, n, k, _ = cases[at]
                gsa.grouped_gemm(a, b, split, m, n, k, recipe, out=outs[s][at], stream=stream)
    torch.cuda.synchronize()
    assert gsa.grouped_gemm_status() == 0
    for o in outs:
        for c, v in zip(cases, o):
            assert np.array_equal(v.double().cpu().numpy(), c[6])
