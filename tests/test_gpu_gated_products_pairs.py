"""The gated products where pairs of blocks take their tiles: against the formulas in 64 bits, the memory that they touch, NaN
in the padding and in single rows, bad splits, graphs with another split, two streams.  Every case says that it is one."""
import numpy as np
import pytest
import torch

from test_gpu_gated_products_more import operand, same_everywhere
from test_gpu_grouped_gemm import MX, NV, dev_split
from test_gpu_grouped_glu import PARAMS, TYPES, U, Case, forward_ref, gradient_ref, gsa_params, near
from test_gpu_moe_bounds import pageable, run  # noqa: F401

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def pairs(m, experts, n):
    """The library's rule: 128 rows an expert and a tile for every two SMs."""
    return m >= 128 * experts and m // 256 * -(-n // 128) >= torch.cuda.get_device_properties(0).multi_processor_count // 2


SHAPES = [([9700, 3, 300], 260, 64, 2), ([0, 5001, 0, 5000, 130], 256, 192, 1), ([20000], 100, 320, 2), ([6500, 129, 255], 257, 1088, 2),
          ([1, 4000, 257, 0, 999], 576, 64, 2)]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("act", sorted(PARAMS))
@pytest.mark.parametrize("split,n,k,groups", SHAPES, ids=str)
def test_forward_and_gradient(recipe, act, split, n, k, groups):
    c = Case(n + k, recipe, split, n, k, groups, 200)
    assert pairs(c.m, len(split), n)
    more = {"act": act, "probs": c.probs, "params": gsa_params(act), "b_groups": groups}
    y, by = forward_ref(c, act)
    dx, bx, dp, bp = gradient_ref(c, act)
    for dtype, last in TYPES.items():
        out = torch.full((c.m, n), float("nan"), dtype=dtype, device="cuda")
        near(gsa.grouped_glu(*c.args(), **more, out=out), y, by, last)
        outs = (torch.full((c.m, 2 * n), float("nan"), dtype=dtype, device="cuda"), torch.full((c.m,), float("nan"), device="cuda"))
        gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more, out=outs)
        near(outs[0], dx, bx, last)
        near(outs[1], dp, bp, U)
        for v in (out, *outs):
            assert bool((v[c.rows:] == 0).all())
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", [([19400, 3, 97], 20, 64), ([9700, 3, 300], 132, 192)], ids=str)
def test_buffers_alone(recipe, split, n, k):
    c, L, e, m = Case(31, recipe, split, n, k, 2), gsa.load(), len(split), sum(split)
    assert pairs(m, e, n)
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
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_nan_stays_in_its_row_and_column(recipe):
    """As in test_gpu_grouped_glu, with rows of both blocks of a pair."""
    rows = 5000
    c = Case(8, recipe, [rows, rows], 150, 256, 2)
    assert pairs(c.m, 2, c.n)
    nan = 0xFF if recipe == MX else 0x7F
    tiles = -(-(c.k // (32 if recipe == MX else 16)) // 4) * 512
    side = -(-c.n // 128) * tiles
    bad = np.zeros((c.m, c.n), bool)
    for row in (5, 200, 4999):   # of expert 1
        c.qa["row_scale"][(-(-rows // 128) + row // 128) * tiles + 16 * (row % 32) + 4 * (row % 128 // 32) + 2] = nan
        bad[rows + row] = True
    c.qb["row_scale"][3 * side + 16 * 7 + 4 * 1] = nan     # expert 1, linear row 39
    c.qb["row_scale"][2 * side + tiles + 16 * 3] = nan     # expert 1, gate row 131
    bad[rows:, [39, 131]] = True
    more = {"act": "clamped_swiglu", "params": gsa_params("clamped_swiglu"), "b_groups": 2, "probs": c.probs}
    y = gsa.grouped_glu(*c.args(), **more, out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(y), bad)
    ref, by = forward_ref(c, "clamped_swiglu")
    assert np.all((np.abs(y - ref) <= by + U * np.abs(ref))[~bad])
    dx, dp = (t.cpu().numpy() for t in gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more, out_dtype=torch.float32))
    ref, bx, _, _ = gradient_ref(c, "clamped_swiglu")
    fine = ~np.concatenate((bad, bad), 1)
    assert np.all((np.abs(dx - ref) <= bx + U * np.abs(ref))[fine])
    assert np.array_equal(np.isnan(dp), bad.any(1))
    assert np.isnan(dx[[rows + 5, rows + 200, rows + 4999]]).all() and gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_bad_splits_write_nothing(recipe):
    rows, n = 5000, 200
    c = Case(15, recipe, [rows, rows], n, 64, 2)
    assert pairs(c.m, 2, n)
    for bad in ([rows, rows + 1], [-1, rows], [1 << 40, 0], [2 * rows, -(1 << 62)]):
        y, dx, dp = (torch.full(s, 5.0, device="cuda") for s in ((c.m, n), (c.m, 2 * n), (c.m,)))
        args = (c.qa, c.qb, dev_split(bad), *c.args()[3:])
        gsa.grouped_glu(*args, b_groups=2, out=y)
        assert gsa.grouped_gemm_status() == 1
        gsa.grouped_glu_bwd(c.dy_dev, *args, b_groups=2, out=(dx, dp))
        assert gsa.grouped_gemm_status() == 1 and gsa.grouped_gemm_status() == 0
        assert bool((y == 5).all()) and bool((dx == 5).all()) and bool((dp == 5).all())


@pytest.mark.parametrize("recipe", [MX, NV])
def test_graph_with_another_split(recipe):
    splits = [[6000, 17, 0, 4064], [1, 4000, 6080, 0], [0, 0, 0, 3], [2500, 2500, 2500, 2581]]
    n, k, m = 136, 192, 10081
    cs = [Case(13 + i, recipe, s, n, k, 2, m - sum(s)) for i, s in enumerate(splits)]
    assert pairs(m, 4, n)
    qa = {"row_data": torch.zeros_like(cs[0].qa["row_data"]), "amax_row": cs[0].qa["amax_row"].clone(),
          "row_scale": torch.zeros(max(c.qa["row_scale"].numel() for c in cs), dtype=torch.uint8, device="cuda")}
    qb, split, dy = {key: v.clone() for key, v in cs[0].qb.items()}, cs[0].dev.clone(), torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    probs = torch.zeros(m, device="cuda")

    def call(stream=None):
        y = gsa.grouped_glu(qa, qb, split, m, n, k, recipe, probs=probs, b_groups=2, out_dtype=torch.float32, stream=stream)
        return (y, *gsa.grouped_glu_bwd(dy, qa, qb, split, m, n, k, recipe, probs=probs, b_groups=2, stream=stream))

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    side = torch.cuda.Stream()
    for c in cs:
        for key, v in c.qa.items():
            qa[key][:v.numel()].copy_(v)
        for key, v in c.qb.items():
            qb[key].copy_(v)
        split.copy_(c.dev)
        dy.copy_(c.dy_dev)
        probs.copy_(c.probs)
        for v in outs:
            v.fill_(float("nan"))
        graph.replay()
        y, by = forward_ref(c, "swiglu")
        dx, bx, dp, bp = gradient_ref(c, "swiglu")
        near(outs[0], y, by, U)
        near(outs[1], dx, bx, 2.0 ** -8)
        near(outs[2], dp, bp, U)
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(u, v) for u, v in zip(got, outs))
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_on_two_streams(recipe):
    """Pairs and single blocks on two streams at once, in opposite orders."""
    cs = [Case(40 + i, recipe, s, n, k, 2) for i, (s, n, k) in enumerate((([9700, 3, 300], 260, 64), ([40, 3, 0, 100], 200, 256), ([2000, 3100], 500, 320)))]
    assert [pairs(c.m, len(c.split), c.n) for c in cs] == [True, False, True]

    def calls(c, stream):
        return (gsa.grouped_glu(*c.args(), b_groups=2, probs=c.probs, stream=stream),
                *gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2, probs=c.probs, stream=stream))

    want = [calls(c, None) for c in cs]
    torch.cuda.synchronize()
    streams, kept = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(20):
        for i in range(len(cs)):
            for s, stream in enumerate(streams):
                at = i if s == 0 else len(cs) - 1 - i
                kept.append((at, calls(cs[at], stream)))
    torch.cuda.synchronize()
    assert gsa.grouped_gemm_status() == 0
    for at, got in kept:
        assert all(torch.equal(u, v) for u, v in zip(got, want[at]))
