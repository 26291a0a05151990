"""The gated products and the products of unquantized rows: memory that they touch, first calls inside captures, two streams
at once, failed launches, and sizes past 32 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split
from test_gpu_grouped_glu import Case, gsa_params
from test_gpu_moe_bounds import bits, pageable, run  # noqa: F401
from test_gpu_moe_error_state import BrokenCapture, qin

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def operand(p, side, m, name):
    return gsa.QIn(p[side], p["s" + side], p[name], m.data.size - 1, m.scale.size)


def same_everywhere():
    first = {}

    def check(o):   # the results do not depend on where the buffers lie
        for k, v in o.items():
            assert np.array_equal(first.setdefault(k, v.copy()), v)
    return check


SHAPES = [([1], 1, 64), ([33, 97, 64, 1, 32], 100, 192), ([300, 17, 0, 64], 320, 576), ([600, 3], 260, 4160)]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", SHAPES, ids=str)
def test_gated_products_touch_their_buffers_alone(recipe, split, n, k):
    c, L, e, m = Case(31, recipe, split, n, k, 2), gsa.load(), len(split), sum(split)
    act = gsa_params("clamped_swiglu")
    inputs = {"a": c.a.data[:-1], "b": c.b.data[:-1], "sa": c.a.scale, "sb": c.b.scale, "amax": c.a.amax, "amaxb": c.b.amax,
              "split": np.array(split, np.int64), "p": c.p}
    dy = c.dy_dev.view(torch.int16).cpu().numpy()
    for code, word in ((gsa.BF16, np.int16), (gsa.FP32, np.int32)):
        run(lambda p: L.gsa_grouped_glu(operand(p, "a", c.a, "amax"), operand(p, "b", c.b, "amaxb"), p["split"], e, m, n, k, recipe, 3, act, p["p"], 2,
                                        p["y"], code, None), inputs, {"y": np.zeros((m, n), word)}, same_everywhere())
        nbytes = L.gsa_grouped_glu_bwd_workspace_size(m, n)
        run(lambda p: L.gsa_grouped_glu_bwd(p["dy"], operand(p, "a", c.a, "amax"), operand(p, "b", c.b, "amaxb"), p["split"], e, m, n, k, recipe, 3, act,
                                            p["p"], 2, p["dx"], code, p["dp"], p["ws"] // 256 * 256 + 256, nbytes, None),
            {**inputs, "dy": dy, "ws": np.zeros(nbytes + 512, np.uint8)}, {"dx": np.zeros((m, 2 * n), word), "dp": np.zeros(m, np.float32)}, same_everywhere())


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", [([1], 1, 64), ([3, 0, 17, 1], 100, 192), ([40, 2], 260, 4160)], ids=str)
def test_products_of_rows_touch_their_buffers_alone(recipe, split, n, k):
    rng, L, e, m = np.random.default_rng(k), gsa.load(), len(split), sum(split)
    b, w = Matrices(rng, [n] * e, k, recipe), Matrices(rng, [n] * (2 * e), k, recipe)
    nbytes = L.gsa_grouped_gemv_workspace_size(e, m, k, recipe)
    for dtype, code, word in ((torch.bfloat16, gsa.BF16, np.int16), (torch.float32, gsa.FP32, np.int32)):
        inputs = {"x": bits(rng, (m, k), dtype), "b": b.data[:-1], "sb": b.scale, "amax": b.amax, "split": np.array(split, np.int64),
                  "ws": np.zeros(nbytes + 512, np.uint8)}
        run(lambda p: L.gsa_grouped_gemv(p["x"], code, operand(p, "b", b, "amax"), p["split"], e, m, n, k, recipe, p["out"], code,
                                         p["ws"] // 256 * 256 + 256, nbytes, None), inputs, {"out": np.zeros((m, n), word)}, same_everywhere())
        inputs.update(b=w.data[:-1], sb=w.scale, amax=w.amax, p=rng.uniform(size=m).astype(np.float32))
        run(lambda p: L.gsa_grouped_glu_gemv(p["x"], code, operand(p, "b", w, "amax"), p["split"], e, m, n, k, recipe, 2, None, p["p"], 2, p["out"], code,
                                             p["ws"] // 256 * 256 + 256, nbytes, None), inputs, {"out": np.zeros((m, n), word)}, same_everywhere())


FIRST = """
import sys
sys.path[:0] = [ROOT, TESTS]
import numpy as np, torch
from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split
from test_gpu_grouped_glu import Case
from nvfp4_quantization_grouped_gb300 import gsa
calls = []
for recipe in (MX, NV):
    for act in ("swiglu", "clamped_swiglu"):
        for rows in (10, 6000):   # single blocks, pairs
            c = Case(3, recipe, [rows, rows], 256, 64, 1)
            calls.append(lambda c=c, act=act: gsa.grouped_glu(*c.args(), act=act))
            calls.append(lambda c=c, act=act: gsa.grouped_glu_bwd(c.dy_dev, *c.args(), act=act)[0])
        x, rng = torch.randn((20, 192), device="cuda"), np.random.default_rng(1)
        b, s = Matrices(rng, [128] * 2, 192, recipe).dev(), dev_split([7, 13])
        calls.append(lambda x=x, b=b, s=s, r=recipe: gsa.grouped_gemv(x, b, s, 128, r))
        w = Matrices(rng, [128] * 4, 192, recipe).dev()
        calls.append(lambda x=x, w=w, s=s, r=recipe, act=act: gsa.grouped_glu_gemv(x, w, s, 128, r, act=act, b_groups=2))
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
    assert r.returncode == 0 and r.stdout.split() == ["same", "24"], r.stdout + r.stderr


@pytest.mark.parametrize("recipe", [MX, NV])
def test_on_two_streams(recipe):
    """All four calls on two streams at once, in opposite orders: workspaces are each call's own."""
    cs = [Case(40 + i, recipe, s, n, k, 2) for i, (s, n, k) in enumerate((([40, 3, 0, 100], 200, 256), ([600, 300], 300, 1024), ([1] * 30, 64, 512)))]
    xs = [torch.randn((c.m, c.k), device="cuda").to(torch.bfloat16) for c in cs]

    def calls(c, x, stream):
        y = gsa.grouped_glu(*c.args(), b_groups=2, probs=c.probs, stream=stream)
        dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2, probs=c.probs, stream=stream)
        z = gsa.grouped_glu_gemv(x, c.qb, c.dev, c.n, recipe, b_groups=2, stream=stream)
        o = gsa.grouped_gemv(x, dict(c.qb, amax_row=c.qb["amax_row"][::2].contiguous()), c.dev, c.n, recipe, out_dtype=torch.float32, stream=stream)
        return y, dx, dp, z, o

    want = [calls(c, x, None) for c, x in zip(cs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    kept = []
    for _ in range(30):
        for i in range(len(cs)):
            for s, stream in enumerate(streams):
                at = i if s == 0 else len(cs) - 1 - i
                kept.append((at, calls(cs[at], xs[at], stream)))
    torch.cuda.synchronize()
    assert gsa.grouped_gemm_status() == 0
    for at, got in kept:
        assert all(torch.equal(u, v) for u, v in zip(got, want[at]))


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("rows", [10, 6000])   # single blocks, pairs
def test_failed_launch_leaves_no_error(recipe, rows):
    c = Case(50, recipe, [rows, rows], 256, 64, 1)
    y, dx, dp = torch.empty((c.m, 256), device="cuda"), torch.empty((c.m, 512), device="cuda"), torch.empty(c.m, device="cuda")
    x, out = torch.randn((c.m, 64), device="cuda"), torch.empty((c.m, 256), device="cuda")
    L = gsa.load()
    n_bwd, n_few = L.gsa_grouped_glu_bwd_workspace_size(c.m, 256), L.gsa_grouped_gemv_workspace_size(2, c.m, 64, recipe)
    ws = torch.empty(max(n_bwd, n_few), dtype=torch.uint8, device="cuda")
    row, t, ts = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), torch.ones((4, 64), device="cuda"), torch.empty((8, 64), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    shape, split = (2, c.m, 256, 64, recipe), c.dev.data_ptr()
    a, b = qin(c.qa, "row"), qin(c.qb, "row")
    with BrokenCapture() as stream:
        for call in (lambda: L.gsa_grouped_glu(a, b, split, *shape, 2, None, None, 1, y.data_ptr(), gsa.FP32, stream),
                     lambda: L.gsa_grouped_glu_bwd(c.dy_dev.data_ptr(), a, b, split, *shape, 2, None, None, 1, dx.data_ptr(), gsa.FP32, dp.data_ptr(),
                                                   ws.data_ptr(), n_bwd, stream),
                     lambda: L.gsa_grouped_gemv(x.data_ptr(), gsa.FP32, b, split, *shape, out.data_ptr(), gsa.FP32, ws.data_ptr(), n_few, stream),
                     lambda: L.gsa_grouped_glu_gemv(x.data_ptr(), gsa.FP32, b, split, *shape, 2, None, None, 1, out.data_ptr(), gsa.FP32, ws.data_ptr(), n_few,
                                                    stream)):
            assert call() == 5
            # a good call on another stream, which looks at the error state behind its launch
            assert L.gsa_moe_permute(t.data_ptr(), None, row.data_ptr(), 4, 2, 64, gsa.FP32, ts.data_ptr(), None, side.cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool((ts == 1).all()) and gsa.grouped_gemm_status() == 0
    assert bool(torch.isfinite(gsa.grouped_glu(*c.args())).all())


@pytest.mark.parametrize("recipe", [MX, NV])
def test_results_past_32_bits(recipe):
    """2^31 and more elements of dx, 2^30 of y: the last rows are those of a call that has them alone."""
    m, n, k, last = 300000, 4096, 64, 300
    c = Case(60, recipe, [last], n, k, 1)
    rows = {"row_data": torch.zeros(m * k // (1 if recipe == MX else 2), dtype=torch.uint8, device="cuda"),
            "row_scale": torch.full((-(-(m - last) // 128) * 512 + c.qa["row_scale"].numel(),), 127 if recipe == MX else 0x38, dtype=torch.uint8, device="cuda"),
            "amax_row": c.qa["amax_row"].repeat(2)}
    rows["row_data"][-c.a.data.size + 1:] = c.qa["row_data"]
    rows["row_scale"][-c.qa["row_scale"].numel():] = c.qa["row_scale"]
    both = {key: torch.cat((v, v)) for key, v in c.qb.items()}
    dy = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    dy[-last:] = c.dy_dev
    split = dev_split([m - last, last])
    y = gsa.grouped_glu(rows, both, split, m, n, k, recipe)
    assert torch.equal(y[-last:], gsa.grouped_glu(*c.args())) and bool((y[:-last] == 0).all())
    del y
    dx, dp = gsa.grouped_glu_bwd(dy, rows, both, split, m, n, k, recipe)
    want = gsa.grouped_glu_bwd(c.dy_dev, *c.args())
    assert torch.equal(dx[-last:], want[0]) and torch.equal(dp[-last:], want[1])
    assert bool((dx[-last - 1000:-last] == 0).all()) and gsa.grouped_gemm_status() == 0


def test_weights_past_32_bits():
    """Codes of 4 GB and more: the last expert's rows are those of a call that has it alone."""
    n, k, e = 16384, 8192, 40
    rng = np.random.default_rng(61)
    b = Matrices(rng, [n], k, MX)
    q = b.dev()
    many = {"row_data": torch.zeros(e * n * k, dtype=torch.uint8, device="cuda"),
            "row_scale": torch.full((e * q["row_scale"].numel(),), 127, dtype=torch.uint8, device="cuda")}
    assert many["row_data"].numel() > 1 << 32
    many["row_data"][-n * k:] = q["row_data"]
    many["row_scale"][-q["row_scale"].numel():] = q["row_scale"]
    x = torch.randn((3, k), device="cuda").to(torch.bfloat16)
    split = dev_split([0] * (e - 1) + [3])
    assert torch.equal(gsa.grouped_gemv(x, many, split, n, MX), gsa.grouped_gemv(x, q, None, n, MX))
    got = gsa.grouped_glu_gemv(x, many, split, n // 2, MX)
    assert torch.equal(got, gsa.grouped_glu_gemv(x, q, None, n // 2, MX)) and gsa.grouped_gemm_status() == 0
