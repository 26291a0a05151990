"""NVFP4 products of operands whose per-expert units are far apart: 1 / S of one side beyond what FP32 holds times a sum,
the other leading back.  Sums are exact in whole units; the scales add one rounding each for 1 / S of either side, and
one each for two multiplications: 4 units of 2^-23, and half a subnormal step."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import NV, Matrices, dev_split, padded

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

PAIRS = [(3e38, 1e-30), (1e-30, 3e38), (3e38, 1e-3), (1e-33, 1e30), (1e30, 1e-33), (2e-33, 4e38 / 2688), (1e20, 1e-20), (3e38, 3e-33)]


def large(m):
    """The same matrices with block scales 2^7 times as large, as the quantizer's are: sums of up to 10^7 units."""
    m.scale = np.where(m.scale == 0x7F, m.scale, m.scale + (7 << 3)).astype(np.uint8)
    m.values = [v * 128 for v in m.values]
    return m


def check(got, a, b):
    for e, (x, w) in enumerate(zip(a.values, b.values)):
        ux, uw = (np.float64(v.amax[e]) / 2688.0 for v in (a, b))
        ref = (np.round(x / ux * 4) @ np.round(w / uw * 4).T) / 16 * ux * uw
        assert np.all(np.abs(ref) < 3e38)
        u = got[e].double().cpu().numpy()
        assert np.all(np.abs(u - ref) <= 4 * 2.0 ** -23 * np.abs(ref) + 2.0 ** -149), PAIRS[e]


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("k", [128, 1024])
def test_product(rows, k):
    rng = np.random.default_rng(rows + k)
    amax_a, amax_b = zip(*PAIRS)
    split, n = [rows] * len(PAIRS), 72
    a, b = large(Matrices(rng, split, k, NV, amax_a)), large(Matrices(rng, [n] * len(PAIRS), k, NV, amax_b))
    got = gsa.grouped_gemm(a.dev(), b.dev(), dev_split(split), sum(split), n, k, NV, out_dtype=torch.float32)
    check(got.split(split), a, b)


@pytest.mark.parametrize("rows", [40, 1000])
def test_weight_gradient(rows):
    rng = np.random.default_rng(rows)
    amax_a, amax_b = zip(*PAIRS)
    split, n, k = [rows] * len(PAIRS), 72, 136
    mp = padded(split, NV)
    a, b = large(Matrices(rng, [n] * len(PAIRS), mp, NV, amax_a)), large(Matrices(rng, [k] * len(PAIRS), mp, NV, amax_b))
    check(gsa.grouped_gemm_wgrad(a.dev("col"), b.dev("col"), dev_split(split), sum(split), n, k, NV), a, b)
