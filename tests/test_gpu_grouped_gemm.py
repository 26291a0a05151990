"""The grouped products of quantized operands against products in 64 bits.

Most cases use operands made of codes and power-of-two scales for which every
partial sum is an integer below 2^24 in a common unit: FP32 sums are then exact
in any order, and the FP32 results must be equal, the BF16 ones equal to their
one rounding.  Padding of the scale tiles holds NaN, which no result may see."""
import numpy as np
import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

MX, NV = gsa.MXFP8, gsa.NVFP4
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_table():
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


E4M3 = e4m3_table()
# E4M3 codes of -6 .. 6 in steps of 1/2 at most, as E2M1's values are: sums stay exact
E4M3_SMALL = np.array([int(np.flatnonzero(E4M3 == v)[0]) for v in E2M1])


def tile_offsets(rows, cols):
    """Byte offset of entry (r, c) of one matrix in scale tiles of 128 x 4, and the tiles' bytes."""
    c4 = -(-cols // 4)
    r, c = np.arange(rows)[:, None], np.arange(cols)[None, :]
    at = (r // 128 * c4 + c // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + c % 4
    return at, -(-rows // 128) * c4 * 512


class Matrices:
    """Quantized [rows_e, k] matrices, one per group, as codes and tiled scales, with their FP64 values."""

    def __init__(self, rng, rows, k, recipe, amax=None):
        b = BLOCK[recipe]
        self.values, data, scale = [], [], []
        self.amax = np.full(len(rows), 2688.0, np.float32) if amax is None else np.asarray(amax, np.float32)
        for e, m in enumerate(rows):
            ke = k[e] if np.ndim(k) else k
            code = rng.integers(0, 16, size=(m, ke))
            power = rng.integers(-1, 2, size=(m, ke // b))
            at, nbytes = tile_offsets(m, ke // b)
            if recipe == MX:
                tiles = np.full(nbytes, 0xFF, np.uint8)
                tiles[at] = power + 127
                data.append(E4M3_SMALL[code].astype(np.uint8).reshape(-1))
            else:
                tiles = np.full(nbytes, 0x7F, np.uint8)
                tiles[at] = (power + 7) << 3
                data.append((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8).reshape(-1))
            scale.append(tiles)
            v = E2M1[code] * np.repeat(2.0 ** power, b, axis=1) if m and ke else np.zeros((m, ke))
            if recipe == NV:
                v = v * (np.float64(self.amax[e]) / 2688.0 if self.amax[e] > 0 else 1.0)
            self.values.append(v)
        self.data, self.scale = np.concatenate(data + [np.zeros(1, np.uint8)]), np.concatenate(scale)
        if self.scale.size == 0:
            self.scale = np.zeros(512 * 64, np.uint8)

    def dev(self, side="row"):
        return {side + "_data": torch.from_numpy(self.data[:-1] if self.data.size > 1 else self.data).cuda(),
                side + "_scale": torch.from_numpy(self.scale).cuda(), "amax_" + side: torch.from_numpy(self.amax).cuda()}


def dev_split(split):
    return torch.tensor(split, dtype=torch.int64, device="cuda")


def rounded(v, dtype):
    return torch.from_numpy(v.astype(np.float32)).to(dtype).double().numpy()


# few rows an expert (single blocks), and many (pairs of blocks on 256 rows), with tiles cut short at every place
SPLITS = [[1], [5, 0, 130], [0, 0, 128, 1, 127, 129, 0], [300, 17, 0, 64], [33, 97, 64, 1, 32], [2] * 40, [0, 0, 0],
          [256], [700, 3, 0, 129], [0, 513, 255, 1, 1000, 31]]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("n,k", [(1, 64), (8, 128), (100, 192), (128, 256), (257, 320), (300, 1024), (512, 576)])
def test_product_exact(recipe, out, split, n, k):
    rng = np.random.default_rng(n * 7 + k + len(split))
    m = sum(split)
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * len(split), k, recipe)
    tail = 3 if n % 2 else 200    # rows that no expert has
    pad = Matrices(rng, [tail], k, recipe)
    qa = a.dev()
    qa["row_data"] = torch.cat((qa["row_data"][:a.data.size - 1], pad.dev()["row_data"]))
    got = gsa.grouped_gemm(qa, b.dev(), dev_split(split), m + tail, n, k, recipe, out_dtype=out,
                           out=torch.full((m + tail, n), float("nan"), dtype=out, device="cuda"))
    assert gsa.grouped_gemm_status() == 0
    ref = np.concatenate([x @ w.T for x, w in zip(a.values, b.values)] + [np.zeros((tail, n))])
    assert np.array_equal(got.double().cpu().numpy(), rounded(ref, out))


def padded(split, recipe):
    b = BLOCK[recipe]
    return [-(-s // b) * b for s in split]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("split", SPLITS + [[1, 15, 16, 17, 31, 33, 47, 63, 65, 255, 257, 1000]], ids=str)
@pytest.mark.parametrize("n,k", [(2, 64), (64, 2), (128, 130), (200, 256), (320, 512)])
def test_wgrad_exact(recipe, out, split, n, k):
    rng = np.random.default_rng(n * 5 + k + len(split))
    mp = padded(split, recipe)
    a, b = Matrices(rng, [n] * len(split), mp, recipe), Matrices(rng, [k] * len(split), mp, recipe)
    got = gsa.grouped_gemm_wgrad(a.dev("col"), b.dev("col"), dev_split(split), sum(split), n, k, recipe, out_dtype=out,
                                 out=torch.full((len(split), n, k), float("nan"), dtype=out, device="cuda"))
    assert gsa.grouped_gemm_status() == 0
    ref = np.stack([x @ w.T for x, w in zip(a.values, b.values)])
    assert np.array_equal(got.double().cpu().numpy(), rounded(ref, out))
    first = rng.integers(-8, 9, size=ref.shape).astype(np.float64)
    acc = torch.from_numpy(first.astype(np.float32)).to("cuda", out)
    gsa.grouped_gemm_wgrad(a.dev("col"), b.dev("col"), dev_split(split), sum(split), n, k, recipe, out=acc,
                           accumulate=True)
    assert np.array_equal(acc.double().cpu().numpy(), rounded(ref + first, out))
