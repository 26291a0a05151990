"""The gated products of many rows an expert, which blocks of a cluster take together, against calls of a few rows each, which
single blocks take: the same sums in the same order, so the same bits.  (Those are tested against 64 bits elsewhere.)"""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, dev_split
from test_gpu_grouped_glu import Case

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

PIECE = 1152   # rows of a call that single blocks take, whatever its other sizes here


def pieces(c, split):
    """The rows of c in calls of one expert's at most PIECE rows: (first row, rows, a, b, groups' index)."""
    tile = 128 * c.k // (1 if c.recipe == MX else 2)
    per = c.qa["row_scale"].numel() // sum(-(-s // 128) for s in split) // 128 * 128   # scale bytes of 128 rows
    bs, bd = (c.qb[k].numel() // len(split) for k in ("row_scale", "row_data"))
    row = scale = 0
    for e, rows in enumerate(split):
        for r in range(0, rows, PIECE):
            n = min(PIECE, rows - r)
            a = {"row_data": c.qa["row_data"][(row + r) * tile // 128:(row + r + n) * tile // 128],
                 "row_scale": c.qa["row_scale"][(scale + r // 128) * per:(scale + -(-(r + n) // 128)) * per]}
            b = {"row_data": c.qb["row_data"][e * bd:(e + 1) * bd], "row_scale": c.qb["row_scale"][e * bs:(e + 1) * bs]}
            if c.recipe == NV:
                a["amax_row"] = c.qa["amax_row"][e:e + 1]
                b["amax_row"] = c.qb["amax_row"].view(len(split), -1)[e].contiguous()
            yield row + r, n, a, b
        row, scale = row + rows, scale + -(-rows // 128)


SPLITS = [([20000], 128, 64), ([20000], 16, 192), ([6000, 0, 7000, 3], 300, 128), ([2000, 1900, 130, 4000, 255, 257], 1000, 192),
          ([5000, 5001], 640, 2112)]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", SPLITS, ids=str)
@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
def test_the_bits_of_single_blocks(recipe, split, n, k, act):
    m, e = sum(split), len(split)
    assert m >= 128 * e and m // 256 * -(-n // 128) >= 76 and PIECE // 256 * -(-n // 128) < 76
    c = Case(70, recipe, split, n, k, 2)
    tail = 300   # rows that no expert has
    rows = m + tail
    x = dict(c.qa, row_data=torch.cat((c.qa["row_data"][:c.a.data.size - 1], c.qa["row_data"][:tail * (k if recipe == MX else k // 2)])))
    probs, dy = torch.cat((c.probs, c.probs[:tail])), torch.cat((c.dy_dev, c.dy_dev[:tail]))
    for dtype in (torch.bfloat16, torch.float32):
        y = gsa.grouped_glu(x, c.qb, c.dev, rows, n, k, recipe, act, probs, b_groups=2, out_dtype=dtype)
        dx, dp = gsa.grouped_glu_bwd(dy, x, c.qb, c.dev, rows, n, k, recipe, act, probs, b_groups=2, out_dtype=dtype)
        only = gsa.grouped_glu_bwd(dy, x, c.qb, c.dev, rows, n, k, recipe, act, probs, b_groups=2, want_dx=False)[1]
        odd = torch.empty(rows * 2 * n + 64, dtype=dtype, device="cuda")[16 // dtype.itemsize:][:rows * 2 * n].view(rows, 2 * n)
        gsa.grouped_glu_bwd(dy, x, c.qb, c.dev, rows, n, k, recipe, act, probs, b_groups=2, want_dprobs=False, out=(odd, None))   # not on 32 bytes
        assert torch.equal(dp, only) and torch.equal(odd, dx)
        for t in (y, dx, dp):
            assert bool((t[m:] == 0).all())
        for at, count, a, b in pieces(c, split):
            one, part = dev_split([count]), slice(at, at + count)
            u = gsa.grouped_glu(a, b, one, count, n, k, recipe, act, probs[part].contiguous(), b_groups=2, out_dtype=dtype)
            du, dpu = gsa.grouped_glu_bwd(dy[part].contiguous(), a, b, one, count, n, k, recipe, act, probs[part].contiguous(), b_groups=2, out_dtype=dtype)
            assert torch.equal(y[part], u) and torch.equal(dx[part], du) and torch.equal(dp[part], dpu), (at, count)
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_a_bad_split_writes_nothing(recipe):
    c = Case(71, recipe, [6000, 6000], 256, 64, 1)
    y = torch.full((c.m, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dp = torch.full((c.m, 512), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((c.m,), 3.0, device="cuda")
    a, b, _, m, n, k, _ = c.args()
    for split in ([6000, 6001], [-1, 6000]):
        gsa.grouped_glu(a, b, dev_split(split), m, n, k, recipe, out=y)
        gsa.grouped_glu_bwd(c.dy_dev, a, b, dev_split(split), m, n, k, recipe, out=(dx, dp))
        assert gsa.grouped_gemm_status() != 0
        assert all(bool((t == 3.0).all()) for t in (y, dx, dp))


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("n", [258, 260, 264, 259])
def test_widths_that_rows_of_other_alignments_have(recipe, n):
    """Rows that start on 4, 8, 16 and 2 bytes, with a last tile of a few columns: the columns of a width of 272 (a multiple
    of 16, on 32 bytes) that has the same weights in front."""
    k, wide, split = 128, 272, [5000, 37, 5600]
    c = Case(72, recipe, split, wide, k, 2)
    m, e = c.m, len(split)
    kb = k if recipe == MX else k // 2
    rows = c.qb["row_data"][:2 * e * wide * kb].view(2 * e, wide, kb)
    b = dict(c.qb, row_data=rows[:, :n].contiguous().view(-1))   # (scale tiles: 3 of 128 rows for either width)
    dy = c.dy_dev[:, :n].contiguous()
    for dtype in (torch.bfloat16, torch.float32):
        y = gsa.grouped_glu(c.qa, c.qb, c.dev, m, wide, k, recipe, "swiglu", c.probs, b_groups=2, out_dtype=dtype)
        got = gsa.grouped_glu(c.qa, b, c.dev, m, n, k, recipe, "swiglu", c.probs, b_groups=2, out_dtype=dtype)
        assert torch.equal(got, y[:, :n])
        padded = torch.zeros((m, wide), dtype=torch.bfloat16, device="cuda")
        padded[:, :n] = dy
        dx, dp = gsa.grouped_glu_bwd(padded, c.qa, c.qb, c.dev, m, wide, k, recipe, "swiglu", c.probs, b_groups=2, out_dtype=dtype)
        du, dpu = gsa.grouped_glu_bwd(dy, c.qa, b, c.dev, m, n, k, recipe, "swiglu", c.probs, b_groups=2, out_dtype=dtype)
        assert torch.equal(du[:, :n], dx[:, :n]) and torch.equal(du[:, n:], dx[:, wide:wide + n]) and torch.equal(dpu, dp)
    assert gsa.grouped_gemm_status() == 0
