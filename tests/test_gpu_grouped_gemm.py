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


@pytest.mark.parametrize("amax", [0.0, 1e-30, 2688.0, 3.4e38])
def test_nvfp4_tensor_scales(amax):
    """1 / (S_A S_B) from the experts' amax, S = 2688 / amax (1 for 0): exact where amax / 2688 is a power of two or the
    quotient is, else within a unit in the last place for each of the divisions and products (4 units of 2^-23)."""
    rng = np.random.default_rng(7)
    split, n, k = [40, 3], 64, 128
    a, b = Matrices(rng, split, k, NV, [amax, 1.5]), Matrices(rng, [n] * 2, k, NV, [2688.0, 21.0])
    got = gsa.grouped_gemm(a.dev(), b.dev(), dev_split(split), 43, n, k, NV, out_dtype=torch.float32).double().cpu().numpy()
    # the sums in whole units first (exact), then the scales: sums that cancel are 0
    ref = []
    for e, (x, w) in enumerate(zip(a.values, b.values)):
        ux, uw = (np.float64(v.amax[e]) / 2688.0 if v.amax[e] > 0 else 1.0 for v in (a, b))
        ref.append((np.round(x / ux * 4) @ np.round(w / uw * 4).T) / 16 * ux * uw)
    ref = np.concatenate(ref)
    with np.errstate(over="ignore"):
        near = np.abs(ref.astype(np.float32).astype(np.float64))
    ok = np.abs(got - ref) <= 4 * 2.0 ** -23 * np.abs(ref) + 2.0 ** -149
    assert np.all(ok | (np.isinf(got) & (near > 1e38)))


@pytest.mark.parametrize("recipe", [MX, NV])
def test_nan_stays_in_its_row_and_column(recipe):
    rng = np.random.default_rng(8)
    split, n, k = [70, 200], 150, 256
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * 2, k, recipe)
    qa, qb = a.dev(), b.dev()
    nan = 0xFF if recipe == MX else 0x7F
    tiles = -(-(k // BLOCK[recipe]) // 4) * 512
    qa["row_scale"][tiles + 16 * 5 + 4 * 1 + 2] = nan              # expert 1, row 37
    qb["row_scale"][2 * tiles + tiles + 16 * 3] = nan              # expert 1, column 128 + 3
    got = gsa.grouped_gemm(qa, qb, dev_split(split), 270, n, k, recipe, out_dtype=torch.float32).cpu().numpy()
    ref = np.concatenate([x @ w.T for x, w in zip(a.values, b.values)])
    bad = np.zeros_like(ref, bool)
    bad[70 + 37] = True
    bad[70:, 131] = True
    assert np.array_equal(np.isnan(got), bad)
    assert np.array_equal(got[~bad].astype(np.float64), ref[~bad])


def decode_copy(q, side, recipe, e_rows, k):
    """FP64 values of each group's matrix from a quantized copy (groups of e_rows[e] rows; k: scalar or per group)."""
    data, scale = q[side + "_data"].cpu().numpy(), q[side + "_scale"].cpu().numpy()
    amax = q["amax_" + side].double().cpu().numpy() if recipe == NV else None
    b, out, d, s = BLOCK[recipe], [], 0, 0
    for e, m in enumerate(e_rows):
        ke = k[e] if np.ndim(k) else k
        at, nbytes = tile_offsets(m, ke // b)
        n = m * ke // (1 if recipe == MX else 2)
        if recipe == MX:
            v = E4M3[data[d:d + n]].reshape(m, ke)
            sc = 2.0 ** (scale[s:s + nbytes][at].astype(np.float64) - 127) if m and ke else np.zeros((m, 0))
        else:
            byte = data[d:d + n].reshape(m, ke // 2)
            v = E2M1[np.stack((byte & 15, byte >> 4), -1).reshape(m, ke)]
            sc = E4M3[scale[s:s + nbytes][at]] if m and ke else np.zeros((m, 0))
            sc = sc * (amax[e] / 2688.0 if amax[e] > 0 else 1.0)
        out.append(v * np.repeat(sc, b, axis=1) if m and ke else np.zeros((m, ke)))
        d, s = d + n, s + nbytes
    return out


@pytest.mark.parametrize("recipe", [MX, NV])
def test_all_three_products_on_quantizer_output(recipe):
    """Forward, input gradient and weight gradient on what the library's own quantizer wrote (tiled scales, NVFP4 with
    the RHT on activations and gradients), against FP64 products of the decoded copies.  FP32 sums of K terms are off
    by at most K 2^-23 of the sum of magnitudes; BF16 results add 2^-8 of their size."""
    rng = np.random.default_rng(9)
    split, n, k = [300, 0, 17, 129], 192, 320
    e, m = len(split), sum(split)

    def bf16(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)

    x, d, w = bf16(m, k), bf16(m, n), bf16(e * n, k)
    rht = recipe == NV
    qx = gsa.fwd(x, None, split, "identity", recipe, rht, 0x1234, scale_layout=gsa.SCALES_TILED)
    qd = gsa.fwd(d, None, split, "identity", recipe, rht, 0x1234, scale_layout=gsa.SCALES_TILED)
    qw = gsa.fwd(w, None, [n] * e, "identity", recipe, scale_layout=gsa.SCALES_TILED)
    s = dev_split(split)
    y = gsa.grouped_gemm(qx, qw, s, m, n, k, recipe)
    dx = gsa.grouped_gemm(qd, qw, s, m, k, n, recipe, b_columnwise=True, out_dtype=torch.float32)
    dw = gsa.grouped_gemm_wgrad(qd, qx, s, m, n, k, recipe)
    assert gsa.grouped_gemm_status() == 0

    def check(got, pairs, terms, rel):
        ref = np.concatenate([a @ b.T for a, b in pairs])
        mass = np.concatenate([np.abs(a) @ np.abs(b).T for a, b in pairs])
        assert np.all(np.abs(got.double().cpu().numpy().reshape(ref.shape) - ref) <= terms * 2.0 ** -23 * mass + rel * np.abs(ref))

    xr, dr = decode_copy(qx, "row", recipe, split, k), decode_copy(qd, "row", recipe, split, n)
    wr, wc = decode_copy(qw, "row", recipe, [n] * e, k), decode_copy(qw, "col", recipe, [k] * e, n)
    mp = padded(split, recipe)
    xc, dc = decode_copy(qx, "col", recipe, [k] * e, mp), decode_copy(qd, "col", recipe, [n] * e, mp)
    check(y, list(zip(xr, wr)), k, 2.0 ** -8)
    check(dx, list(zip(dr, wc)), n, 2.0 ** -22)
    check(dw, list(zip(dc, xc)), max(mp), 2.0 ** -22)


@pytest.mark.parametrize("recipe", [MX, NV])
def test_weight_gradient_against_differences(recipe):
    """loss = sum(G * product(A, B)) is linear in B: the loss of B' minus that of B is <dW, B' - B>.  All operands are
    integers in a common unit and all sums below 2^53 of it, so both sides are equal."""
    rng = np.random.default_rng(10)
    split, n, k = [64, 32, 0, 96], 64, 128
    e, m, b = len(split), sum(split), BLOCK[recipe]

    def copies(code, split):
        """Row and column copies (scales 1) of codes [M, C] grouped by split (multiples of the block)."""
        row, col = code, np.concatenate([c.T.reshape(-1) for c in np.split(code, np.cumsum(split)[:-1])])
        q = {}
        for side, c in (("row", row.reshape(-1)), ("col", col)):
            byte = E4M3_SMALL[c].astype(np.uint8) if recipe == MX else (c[0::2] | c[1::2] << 4).astype(np.uint8)
            q[side + "_data"] = torch.from_numpy(byte).cuda()
            q[side + "_scale"] = torch.full((1 << 16,), 127 if recipe == MX else 0x38, dtype=torch.uint8, device="cuda")
            q["amax_" + side] = torch.full((len(split),), 2688.0, device="cuda")
        return q

    assert all(s % b == 0 for s in split)
    a, g = rng.integers(0, 16, (m, k)), rng.integers(0, 16, (m, n))
    w = [rng.integers(0, 16, (e * n, k)) for _ in range(2)]
    s, qa = dev_split(split), copies(a, split)
    loss = [float((gsa.grouped_gemm(qa, copies(v, [n] * e), s, m, n, k, recipe, out_dtype=torch.float32).double() *
                   torch.from_numpy(E2M1[g]).cuda()).sum()) for v in w]
    dw = gsa.grouped_gemm_wgrad(copies(g, split), qa, s, m, n, k, recipe).double().cpu().numpy().reshape(e * n, k)
    assert loss[1] - loss[0] == float(np.sum(dw * (E2M1[w[1]] - E2M1[w[0]])))


def test_bad_device_split_is_reported_and_nothing_is_written():
    rng = np.random.default_rng(11)
    split, n, k = [10, 20], 64, 128
    a, b = Matrices(rng, split, k, MX), Matrices(rng, [n] * 2, k, MX)
    ac, bc = Matrices(rng, [n] * 2, padded(split, MX), MX), Matrices(rng, [k] * 2, padded(split, MX), MX)
    for bad in ([10, 21], [-1, 20], [2 ** 40, 1], [31, -1]):
        out = torch.full((30, n), 7.0, dtype=torch.float32, device="cuda")
        gsa.grouped_gemm(a.dev(), b.dev(), dev_split(bad), 30, n, k, MX, out=out)
        assert gsa.grouped_gemm_status() == 1 and gsa.grouped_gemm_status() == 0
        assert bool((out == 7.0).all())
        dw = torch.full((2, n, k), 7.0, dtype=torch.float32, device="cuda")
        gsa.grouped_gemm_wgrad(ac.dev("col"), bc.dev("col"), dev_split(bad), 30, n, k, MX, out=dw)
        assert gsa.grouped_gemm_status() == 1 and bool((dw == 7.0).all())
    # more scale tiles than the buffer holds: 30 single rows, one tile
    many, short = dev_split([1] * 30), a.dev()
    short["row_scale"] = short["row_scale"][:512].contiguous()
    b30 = Matrices(rng, [n] * 30, k, MX)
    gsa.grouped_gemm(short, b30.dev(), many, 30, n, k, MX)
    assert gsa.grouped_gemm_status() == 1
    got = gsa.grouped_gemm(a.dev(), b.dev(), dev_split(split), 30, n, k, MX, out_dtype=torch.float32)
    assert gsa.grouped_gemm_status() == 0
    assert np.array_equal(got.double().cpu().numpy(), np.concatenate([x @ w.T for x, w in zip(a.values, b.values)]))


@pytest.mark.parametrize("recipe", [MX, NV])
def test_graph_replay_with_another_split_and_another_stream(recipe):
    """One capture, replayed after the split changed in place; and the calls on a stream of their own."""
    rng = np.random.default_rng(12)
    n, k, m = 96, 192, 300
    splits = [[100, 0, 200], [31, 169, 100]]
    s = dev_split(splits[0])
    a = [Matrices(rng, v, k, recipe) for v in splits]
    b = Matrices(rng, [n] * 3, k, recipe)
    size = max(v.scale.size for v in a)

    def dev_a(v):
        q = v.dev()
        q["row_scale"] = torch.cat((q["row_scale"], torch.zeros(size - v.scale.size, dtype=torch.uint8, device="cuda")))
        return q

    qa, qb = dev_a(a[0]), b.dev()
    gsa.grouped_gemm(qa, qb, s, m, n, k, recipe)   # first call outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gsa.grouped_gemm(qa, qb, s, m, n, k, recipe, out_dtype=torch.float32)
    for i in (0, 1):
        for key, v in dev_a(a[i]).items():
            qa[key].copy_(v)
        s.copy_(dev_split(splits[i]))
        graph.replay()
        ref = np.concatenate([x @ w.T for x, w in zip(a[i].values, b.values)])
        assert np.array_equal(out.double().cpu().numpy(), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gsa.grouped_gemm(qa, qb, s, m, n, k, recipe, out_dtype=torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out) and gsa.grouped_gemm_status(side) == 0


@pytest.mark.parametrize("recipe", [MX, NV])
def test_wgrad_graph_and_determinism(recipe):
    rng = np.random.default_rng(13)
    split, n, k = [500, 17, 0, 48, 300], 192, 320
    mp = padded(split, recipe)
    a, b = Matrices(rng, [n] * 5, mp, recipe), Matrices(rng, [k] * 5, mp, recipe)
    qa, qb, s = a.dev("col"), b.dev("col"), dev_split(split)
    first = gsa.grouped_gemm_wgrad(qa, qb, s, sum(split), n, k, recipe)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gsa.grouped_gemm_wgrad(qa, qb, s, sum(split), n, k, recipe)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, first)


@pytest.mark.parametrize("recipe", [MX, NV])
def test_no_rows_at_all(recipe):
    """Zero rows: an empty product, and zero weight gradients from empty copies."""
    x, s = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), dev_split([0, 0])
    q = gsa.fwd(x, None, [0, 0], "identity", recipe, scale_layout=gsa.SCALES_TILED)
    w = Matrices(np.random.default_rng(1), [64, 64], 64, recipe).dev()
    assert gsa.grouped_gemm(q, w, s, 0, 64, 64, recipe).shape == (0, 64)
    dw = gsa.grouped_gemm_wgrad(q, q, s, 0, 64, 64, recipe, out=torch.full((2, 64, 64), 5.0, device="cuda"))
    assert bool((dw == 0).all()) and gsa.grouped_gemm_status() == 0
    gsa.grouped_gemm_wgrad(q, q, s, 0, 64, 64, recipe, out=dw.fill_(5.0), accumulate=True)
    assert bool((dw == 5.0).all())


def test_python_refusals():
    rng = np.random.default_rng(14)
    a, b, s = Matrices(rng, [4, 4], 64, NV).dev(), Matrices(rng, [64, 64], 64, NV).dev(), dev_split([4, 4])
    for call in (lambda: gsa.grouped_gemm({}, b, s, 8, 64, 64, NV), lambda: gsa.grouped_gemm(a, {}, s, 8, 64, 64, NV),
                 lambda: gsa.grouped_gemm(a, b, s.int(), 8, 64, 64, NV),
                 lambda: gsa.grouped_gemm(a, b, s.cpu(), 8, 64, 64, NV),
                 lambda: gsa.grouped_gemm(a, b, s, 8, 64, 64, NV, out_dtype=torch.float16),
                 lambda: gsa.grouped_gemm(a, b, s, 8, 64, 96, NV), lambda: gsa.grouped_gemm(a, b, s, 9, 64, 64, NV),
                 lambda: gsa.grouped_gemm(a, b, s, 8, 65, 64, NV), lambda: gsa.grouped_gemm(a, b, s, 8, 64, 64, 2),
                 lambda: gsa.grouped_gemm(dict(a, amax_row=a["amax_row"][:1]), b, s, 8, 64, 64, NV),
                 lambda: gsa.grouped_gemm(a, b, s, 8, 64, 64, NV, out=torch.empty((8, 32), device="cuda")),
                 lambda: gsa.grouped_gemm(a, b, s, 8, 64, 64, NV, b_columnwise=True),
                 lambda: gsa.grouped_gemm_wgrad(a, b, s, 8, 64, 64, NV),
                 lambda: gsa.grouped_gemm_wgrad(Matrices(rng, [64] * 2, 16, NV).dev("col"),
                                                Matrices(rng, [64] * 2, 16, NV).dev("col"), s, 8, 64, 64, NV,
                                                accumulate=True)):
        with pytest.raises(gsa.GsaError):
            call()


@pytest.mark.parametrize("recipe", [MX, NV])
def test_ffn_example(recipe):
    """The example's step (sort, gather, both projections, activation, way back, all gradients).  Each quantized operand
    is within 2^-4 (E4M3) or 2^-2 (E2M1, plus 2^-4 of its scale) of itself element by element.  The results go through up
    to seven of them (the squared activation counts twice), whose errors are independent: they add in quadrature."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_ffn.py")
    spec = importlib.util.spec_from_file_location("moe_ffn", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    e, t, topk, hidden, width = 6, 500, 2, 192, 256

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    w1, w2 = normal(e, width, hidden, scale=hidden ** -0.5), normal(e, hidden, width, scale=width ** -0.5)
    x, dout = normal(t, hidden), normal(t, hidden)
    probs, idx = torch.topk(torch.softmax(torch.randn((t, e), generator=g, device="cuda"), 1), topk)
    idx[::7, 1] = -1    # dropped slots
    idx[3] = -1         # a token that no expert takes
    ffn = ex.MoeFfn(w1, w2, "srelu", recipe)
    out, saved = ffn.forward(x, idx, probs)
    got = (out, *ffn.backward(dout, saved))
    assert gsa.grouped_gemm_status() == 0
    one = 2.0 ** -4 if recipe == MX else 2.0 ** -2 + 2.0 ** -4
    for name, u, v, operands in zip(("out", "dx", "dprobs", "dw1", "dw2"), got, ex.reference(x, idx, probs, w1, w2, dout, "srelu"),
                                    (6, 7, 6, 6, 5)):
        err = float((u.float() - v).norm() / v.norm())
        assert err <= operands ** 0.5 * one, (name, err)
    assert bool((got[0][3] == 0).all()) and bool((got[1][3] == 0).all()) and bool((got[2][idx < 0] == 0).all())
