"""Long sums of the grouped products.

The tensor core cuts its FP32 sums off toward zero at every step, so an FP32
result longer than 16 stages of 128 bytes is taken in pieces that are added in
FP32 with rounding.  First sums that are exact in any order, at lengths around
the pieces' ends; then sums of one sign, whose error would otherwise grow with
their length."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import BLOCK, E2M1, E4M3, MX, NV, Matrices, dev_split, padded, rounded, tile_offsets

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(40, 24), (300, 264)])
def test_wgrad_exact_around_the_pieces(recipe, out, n, k):
    rng = np.random.default_rng(n)
    split = [s * (1 if recipe == MX else 2) for s in (2047, 2048, 2049, 0, 2176, 4097, 100, 6200)]
    mp = padded(split, recipe)
    a, b = Matrices(rng, [n] * len(split), mp, recipe), Matrices(rng, [k] * len(split), mp, recipe)
    got = gsa.grouped_gemm_wgrad(a.dev("col"), b.dev("col"), dev_split(split), sum(split), n, k, recipe, out_dtype=out)
    assert gsa.grouped_gemm_status() == 0
    ref = np.stack([x @ w.T for x, w in zip(a.values, b.values)])
    assert np.array_equal(got.double().cpu().numpy(), rounded(ref, out))


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split", [[40, 3, 0, 100], [600, 300]], ids=str)
@pytest.mark.parametrize("k", [2048, 2112, 4096, 4160, 8256])
def test_product_exact_around_the_pieces(recipe, split, k):
    rng = np.random.default_rng(k)
    n = 200
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * len(split), k, recipe)
    got = gsa.grouped_gemm(a.dev(), b.dev(), dev_split(split), sum(split), n, k, recipe, out_dtype=torch.float32)
    assert gsa.grouped_gemm_status() == 0
    ref = np.concatenate([x @ w.T for x, w in zip(a.values, b.values)])
    assert np.array_equal(got.double().cpu().numpy(), rounded(ref, torch.float32))


def positive(rng, rows, k, recipe):
    """One quantized [rows, k] matrix of positive values with scales of many sizes: (codes, tiles), its FP64 values."""
    b = BLOCK[recipe]
    at, nbytes = tile_offsets(rows, k // b)
    if recipe == MX:
        code, scale = rng.integers(0x30, 0x48, size=(rows, k)), rng.integers(124, 131, size=(rows, k // b))
        v, s, data = E4M3[code], 2.0 ** (scale - 127), code
    else:
        code, scale = rng.integers(1, 8, size=(rows, k)), rng.integers(0x20, 0x58, size=(rows, k // b))
        v, s, data = E2M1[code], E4M3[scale], code[:, 0::2] | code[:, 1::2] << 4
    tiles = np.full(nbytes, 0x7F, np.uint8)
    tiles[at] = scale
    return data.astype(np.uint8).reshape(-1), tiles, v * np.repeat(s, b, axis=1)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("op", ["product", "wgrad"])
def test_error_does_not_grow_with_the_length(recipe, op):
    """A piece of FP32 results is 64 steps of 32 bytes.  A step cuts off less than a unit in the last place of the running
    sum, 2^-23 of it at most: over a growing sum (64 + 1) / 2 units.  The 16 or 32 pieces are added with 2^-24 each: 16
    units.  In all 49 units of 2^-23."""
    rng = np.random.default_rng(5)
    length, n, k = 65536, 96, 72
    da, sa, va = positive(rng, n, length, recipe)
    db, sb, vb = positive(rng, k, length, recipe)
    side = "col" if op == "wgrad" else "row"
    amax = torch.full((1,), 2688.0, device="cuda")
    qa, qb = ({side + "_data": torch.from_numpy(d).cuda(), side + "_scale": torch.from_numpy(s).cuda(), "amax_" + side: amax}
              for d, s in ((da, sa), (db, sb)))
    if op == "wgrad":
        got = gsa.grouped_gemm_wgrad(qa, qb, dev_split([length]), length, n, k, recipe, out_dtype=torch.float32)[0]
    else:
        got = gsa.grouped_gemm(qa, qb, dev_split([n]), n, k, length, recipe, out_dtype=torch.float32)
    assert gsa.grouped_gemm_status() == 0
    ref = va @ vb.T
    assert np.max(np.abs(got.double().cpu().numpy() / ref - 1)) <= 49 * 2.0 ** -23
