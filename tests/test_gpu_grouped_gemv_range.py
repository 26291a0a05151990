"""Products of a few rows whose values and weights are far from 1, one side large and the other small, so that the results are
ordinary: nothing on the way leaves FP32's range where the result does not.  Bounds as in test_gpu_grouped_gemv; a sum that
ends in the subnormal range loses at most one of its steps with each 32 bytes of k."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split
from test_gpu_grouped_gemv import TYPES, close, mass_bound
from test_gpu_grouped_glu import U

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def moved(m, recipe, group, power):
    """Group `group` of the matrices times 2^power: block scales (MXFP8), or amax."""
    if recipe == MX:
        per = m.scale.size // len(m.values)
        s = m.scale[group * per:(group + 1) * per]
        to = s.astype(np.int64) + power
        assert np.all((s == 0xFF) | ((to >= 0) & (to < 0xFF)))
        s[:] = np.where(s == 0xFF, s, to).astype(np.uint8)
    else:
        m.amax[group] *= 2.0 ** power
    m.values[group] = m.values[group] * 2.0 ** power


# powers of two of rows and weights (NVFP4: amax up to 2^127, 2688 units)
FAR = {MX: [(-110, 122), (-126, 124), (-30, 115), (-60, 118), (-41, 124), (-39, 120), (-100, 100), (100, -110), (120, -120), (0, -120), (-20, -115), (3, 112)],
       NV: [(-110, 115), (-120, 110), (-30, 110), (-60, 115), (-100, 100), (100, -110), (120, -115), (0, -100), (-20, -100), (3, 110)]}


def rows_of(rng, count, k, power, dtype):
    v = rng.standard_normal((count, k)) * 2.0 ** power
    v[1::2] *= 2.0 ** rng.integers(-9, 1, size=v[1::2].shape)
    return torch.from_numpy(v).to(dtype)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("dtype", [t for t in TYPES if t is not torch.float16], ids=str)
@pytest.mark.parametrize("k", [64, 1088])
def test_products(recipe, dtype, k):
    rng, far, n = np.random.default_rng(k), FAR[recipe], 40
    b = Matrices(rng, [n] * len(far), k, recipe)
    for e, (_, power) in enumerate(far):
        moved(b, recipe, e, power)
    x = torch.cat([rows_of(rng, 5, k, power, dtype) for power, _ in far]).cuda()
    got = gsa.grouped_gemv(x, b.dev(), dev_split([5] * len(far)), n, recipe, out_dtype=torch.float32).double().cpu().numpy()
    for e, w in enumerate(b.values):
        v = x[5 * e:5 * e + 5].double().cpu().numpy()
        ref = v @ w.T
        assert np.max(np.abs(ref)) < 2.0 ** 127
        bound = mass_bound(v, w, k, recipe) + 3 * 2.0 ** -23 * np.abs(ref) + (k / 32 + 8) * 2.0 ** -149
        assert close(got[5 * e:5 * e + 5], ref, bound, torch.float32), far[e]
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_gated(recipe):
    """Gate and linear rows of about the rows' reciprocal size.  g and u are off by their products' bounds; y = g s u moves by
    |u| (s + |g| s q) of g's and |g| s of u's, twice that covers the second order (the bounds are below 2^-10 of g), and
    the activation adds (16 + 3 |z|) U of y."""
    rng, far, n, k = np.random.default_rng(5), [f for f in FAR[recipe] if abs(sum(f)) <= 20 and f[0] < 118], 40, 192   # (scales of 2^-127 at least)
    b = Matrices(rng, [n] * (2 * len(far)), k, recipe)
    for e, (row, _) in enumerate(far):
        for side in (0, 1):
            moved(b, recipe, 2 * e + side, -row - 8)
    x = torch.cat([rows_of(rng, 5, k, power, torch.float32) for power, _ in far]).cuda()
    got = gsa.grouped_glu_gemv(x, b.dev(), dev_split([5] * len(far)), n, recipe, b_groups=2).double().cpu().numpy()
    for e in range(len(far)):
        v = x[5 * e:5 * e + 5].double().cpu().numpy()
        (g, bg), (u, bu) = ((v @ w.T, mass_bound(v, w, k, recipe) + 3 * 2.0 ** -23 * np.abs(v @ w.T)) for w in b.values[2 * e:2 * e + 2])
        s = 1 / (1 + np.exp(-g))
        ref = g * s * u
        bound = 2 * (np.abs(u) * (s + np.abs(g) * s * (1 - s)) * bg + np.abs(g) * s * bu) + (16 + 3 * np.abs(g)) * U * np.abs(ref) + 2.0 ** -120
        assert close(got[5 * e:5 * e + 5], ref, bound, torch.float32), far[e]
    assert gsa.grouped_gemm_status() == 0
