"""Products of a few unquantized rows with quantized weights, plain and gated, against their formulas in 64 bits.

Rows of small integers give sums that are exact in FP32 in any order: FP32 results must be equal, others equal to their one
rounding.  Rows of any values: a row's eight digits are sums of their own, each off by at most (K / 16 + 16) units of 2^-23 of
its sum of magnitudes (a unit a step, and for each of the last sums).  A digit is the code nearest to what the one before
leaves, which is at most a third of the block's largest value, then an eighth of that and so on: the digits' magnitudes are
at most |x| and the block's largest value together.  What eight digits leave is half of 2^-20 in a unit in which the
largest value of the block is 3 at least: 2^-22 of it; and for blocks so far below the row's largest value that their scale
stops at 2^-17 of its, 2^-39 of that value."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, dev_split, rounded
from test_gpu_grouped_glu import PARAMS, U, gsa_params

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

TYPES = [torch.bfloat16, torch.float16, torch.float32]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
# below 2^-14 an FP16 result is a multiple of 2^-24: half of it
SMALL = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
SPLITS = [[1], [3], [1, 0, 2], [0, 0, 8, 1, 9, 0], [5, 16, 0, 17], [1] * 40, [0, 0, 0], [33, 0, 64, 7], [2] + [0] * 254 + [1]]
SHAPES = [(1, 64), (8, 128), (17, 192), (100, 320), (128, 1024), (129, 576), (200, 4096), (1111, 1088)]


def ids(v):
    return str(v) if len(str(v)) < 40 else "%d experts" % len(v)


def mass_bound(x, w, k, recipe):
    """Of x w^T before the last rounding (x [m, k], w [n, k] in FP64)."""
    ax, aw, b = np.abs(x), np.abs(w), 32 if recipe == MX else 16
    top = np.repeat(ax.reshape(len(x), -1, b).max(2), b, 1)
    largest = ax.max(1, initial=0.0)[:, None] * aw.max(1, initial=0.0)[None, :]
    return (k / 16 + 16) * 2.0 ** -23 * ((ax + top) @ aw.T) + 2.0 ** -22 * (top @ aw.T) + k * 2.0 ** -39 * largest


# from here on rounding to the nearest gives infinity: half a step above the type's largest value
ENDS = {torch.bfloat16: (2 - 2.0 ** -8) * 2.0 ** 127, torch.float16: 65520.0, torch.float32: (2 - 2.0 ** -24) * 2.0 ** 127}


def close(got, ref, bound, out):
    """Within the bound and the last rounding; infinite with the right sign where that goes past the type's end."""
    over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + bound >= ENDS[out])
    with np.errstate(invalid="ignore"):
        return np.all(over | (np.abs(got - ref) <= bound + HALF[out] * (np.abs(ref) + bound) + SMALL[out]))


def by_expert(x, split, f, n):
    """f(e, rows of expert e) put together, zeros for the rows that no expert has."""
    out, r = np.zeros((x.shape[0], n)), 0
    for e, m in enumerate(split):
        if m:
            out[r:r + m] = f(e, x[r:r + m])
        r += m
    return out


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split", SPLITS, ids=ids)
@pytest.mark.parametrize("n,k", SHAPES)
def test_exact(recipe, split, n, k):
    """Integers of -3 .. 3: every partial sum is a multiple of 1/4 below 2^22."""
    if len(split) > 100 and n * k > 10000:
        n, k = 40, 192
    rng = np.random.default_rng(n * 3 + k + len(split))
    rows, tail = sum(split), n % 4
    b = Matrices(rng, [n] * len(split), k, recipe)
    x = rng.integers(-3, 4, size=(rows + tail, k)).astype(np.float64)
    ref = by_expert(x, split, lambda e, v: v @ b.values[e].T, n)
    qb, s = b.dev(), dev_split(split)
    for dtype in TYPES:
        xd = torch.from_numpy(x).cuda().to(dtype)
        for out in {dtype, torch.float32}:
            got = gsa.grouped_gemv(xd, qb, s, n, recipe, out=torch.full((rows + tail, n), float("nan"), dtype=out, device="cuda"))
            assert np.array_equal(got.double().cpu().numpy(), rounded(ref, out))
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("split", SPLITS, ids=ids)
@pytest.mark.parametrize("n,k", SHAPES)
def test_any_values(recipe, dtype, split, n, k):
    """Normal rows, some of them with values of many sizes."""
    if len(split) > 100 and n * k > 10000:
        n, k = 40, 192
    rng = np.random.default_rng(n + k + len(split))
    rows = sum(split)
    amax = 2.0 ** rng.uniform(-6, 6, len(split)) * 2688
    b = Matrices(rng, [n] * len(split), k, recipe, amax if recipe == NV else None)
    v = rng.standard_normal((rows, k))
    v[::3] *= 2.0 ** rng.integers(-12, 5, size=v[::3].shape)
    x = torch.from_numpy(v).cuda().to(dtype)
    v = x.double().cpu().numpy()
    ref = by_expert(v, split, lambda e, w: w @ b.values[e].T, n)
    bound = by_expert(v, split, lambda e, w: mass_bound(w, b.values[e], k, recipe) + 3 * 2.0 ** -23 * np.abs(w @ b.values[e].T), n)
    for out in {dtype, torch.float32}:
        got = gsa.grouped_gemv(x, b.dev(), dev_split(split), n, recipe, out_dtype=out).double().cpu().numpy()
        assert close(got, ref, bound, out)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("act", sorted(PARAMS))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("split", SPLITS, ids=ids)
@pytest.mark.parametrize("n,k,groups", [(1, 64, 2), (100, 192, 2), (128, 1024, 1), (129, 320, 2), (256, 4096, 1)])
def test_gated(recipe, act, dtype, split, n, k, groups):
    """y = p act(g, u): g and u off by the bound of a plain product, the activation by that of grouped_glu.  d act / d g is at
    most 1.1 max(1, alpha) |b|, d act / d u at most |a s|."""
    if len(split) > 100 and n * k > 10000:
        n, k, groups = 40, 192, 2
    rng = np.random.default_rng(n + k + len(split))
    rows = sum(split)
    b = Matrices(rng, [2 * n // groups] * (groups * len(split)), k, recipe)
    x = torch.from_numpy(rng.standard_normal((rows, k)) * 0.25 / np.sqrt(k)).cuda().to(dtype)
    v = x.double().cpu().numpy()
    p = rng.uniform(-1, 1, rows).astype(np.float32)
    weights = [np.concatenate(b.values[e * groups:(e + 1) * groups]) for e in range(len(split))]
    h = by_expert(v, split, lambda e, w: w @ weights[e].T, 2 * n)
    off = by_expert(v, split, lambda e, w: mass_bound(w, weights[e], k, recipe) + 3 * 2.0 ** -23 * np.abs(w @ weights[e].T), 2 * n)
    limit, alpha, add = PARAMS[act]
    a, lin = np.minimum(h[:, :n], limit), np.clip(h[:, n:], -limit, limit) + add
    z = alpha * a
    s = 1 / (1 + np.exp(-z))
    more = {"act": act, "params": gsa_params(act), "b_groups": groups}
    for scale, probs in ((1.0, None), (p[:, None].astype(np.float64), torch.from_numpy(p).cuda())):
        ref = a * s * lin * scale
        bound = np.abs(scale) * (1.1 * max(1, alpha) * (np.abs(lin) + off[:, n:]) * off[:, :n] + np.abs(a * s) * off[:, n:] +
                                 (16 + 3 * np.abs(z)) * U * np.abs(a * s) * (np.abs(lin) + 4 * add)) + 2.0 ** -120
        for out in {dtype, torch.float32}:
            got = gsa.grouped_glu_gemv(x, b.dev(), dev_split(split), n, recipe, probs=probs, out_dtype=out, **more).double().cpu().numpy()
            assert close(got, ref, bound, out)
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_rows_across_the_range(recipe, dtype):
    """Rows near the largest and the smallest values of their type, and rows whose values span all of it."""
    rng = np.random.default_rng(20)
    n, k = 70, 256
    sizes = np.array([2.0 ** 120, 2.0 ** 60, 2.0 ** -60, 2.0 ** -118, 2.0 ** -130, 1.0])
    b = Matrices(rng, [n], k, recipe, [2688.0])
    v = rng.standard_normal((8, k))
    v[:6] *= sizes[:, None]
    v[6] *= 2.0 ** np.linspace(-126, 100, k)
    v[7] = 0.0
    x = torch.from_numpy(v).cuda().to(dtype)
    v = x.double().cpu().numpy()
    ref, w = v @ b.values[0].T, b.values[0]
    got = gsa.grouped_gemv(x, b.dev(), None, n, recipe, out_dtype=torch.float32).double().cpu().numpy()
    bound = mass_bound(v, w, k, recipe) + U * np.abs(ref) + 2.0 ** -126 * (np.abs(ref) < 2.0 ** -125)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("amax", [0.0, 1e-30, 1e30, 3.4e38])
def test_nvfp4_tensor_scales(amax):
    """Units far out with rows leading back: 1 / S is off by 2 units of 2^-23, its products by one each."""
    rng = np.random.default_rng(21)
    n, k = 40, 192
    b = Matrices(rng, [n], k, NV, [amax])
    unit = np.float64(b.amax[0]) / 2688.0 if amax else 1.0
    codes = np.round(b.values[0] / unit * 4) / 4
    for size in (1.0, 2.0 ** -100, 2.0 ** 100):
        v = rng.integers(-3, 4, size=(5, k)) * size
        ref = (v / size @ codes.T) * unit * size
        x = torch.from_numpy(v).cuda().float()
        got = gsa.grouped_gemv(x, b.dev(), None, n, NV).double().cpu().numpy()
        fits = np.abs(ref) < 3e38
        assert np.all(np.abs(got - ref)[fits] <= (4 * 2.0 ** -23 * np.abs(ref) + 2.0 ** -148)[fits])
        assert np.all(np.abs(got[~fits]) > 3e38)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_infinities_and_nan(recipe, dtype):
    """Infinite and NaN values of a row, and NaN scales of a weight row, do what products and sums do with them, in their row
    and column alone."""
    rng = np.random.default_rng(22)
    n, k, nan = 150, 192, 0xFF if recipe == MX else 0x7F
    b = Matrices(rng, [n], k, recipe)
    v = rng.integers(-3, 4, size=(6, k)).astype(np.float64)
    v[1, 5], v[2, 70], v[3, 100], v[4, 7], v[4, 150] = np.inf, -np.inf, np.nan, np.inf, np.inf
    b.scale[16 * 9 + 4 * 2 + 1] = nan     # row 73, in its second block
    w = b.values[0].copy()
    block = 32 if recipe == MX else 16
    w[73, block:2 * block] = np.nan
    with np.errstate(invalid="ignore"):
        ref = (v[:, None, :] * w[None, :, :]).sum(2)
    x = torch.from_numpy(v).cuda().to(dtype)
    got = gsa.grouped_gemv(x, b.dev(), None, n, recipe, out_dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert np.array_equal(got[fine], ref[fine])
    many = torch.ones((3, k), dtype=dtype, device="cuda")
    many[1, :9] = float("inf")    # more than eight: NaN, whatever the weights
    many[2, 10:18] = float("-inf")
    got = gsa.grouped_gemv(many, b.dev(), None, n, recipe, out_dtype=torch.float32).double().cpu().numpy()
    assert np.isfinite(got[0][np.arange(n) != 73]).all() and np.isnan(got[1]).all()
    with np.errstate(invalid="ignore"):
        ref = (many[2].double().cpu().numpy() * w).sum(1)
    assert np.array_equal(np.isnan(got[2]), np.isnan(ref)) and np.array_equal(got[2][~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("recipe", [MX, NV])
def test_rows_do_not_depend_on_their_number(recipe):
    """A row's result is the same bits alone and among others, whatever expert's turn it is."""
    rng = np.random.default_rng(23)
    n, k = 300, 2112
    b = Matrices(rng, [n], k, recipe)
    x = torch.from_numpy(rng.standard_normal((40, k))).cuda().to(torch.bfloat16)
    q = b.dev()
    whole = gsa.grouped_gemv(x, q, None, n, recipe, out_dtype=torch.float32)
    for r0, r1 in ((0, 1), (3, 5), (7, 10), (8, 16), (9, 26), (39, 40)):
        assert torch.equal(gsa.grouped_gemv(x[r0:r1].clone(), q, None, n, recipe, out_dtype=torch.float32), whole[r0:r1])


@pytest.mark.parametrize("recipe", [MX, NV])
def test_graph_stream_and_views(recipe):
    """Captured, replayed with another split in place; on another stream; out inside a larger tensor."""
    rng = np.random.default_rng(24)
    n, k, experts = 136, 320, 5
    b = Matrices(rng, [n] * experts, k, recipe)
    x = rng.integers(-3, 4, size=(12, k)).astype(np.float64)
    xd, qb, s = torch.from_numpy(x).cuda().to(torch.bfloat16), b.dev(), dev_split([2, 0, 5, 1, 4])
    graph = torch.cuda.CUDAGraph()
    gsa.grouped_gemv(xd, qb, s, n, recipe)
    with torch.cuda.graph(graph):
        out = gsa.grouped_gemv(xd, qb, s, n, recipe, out_dtype=torch.float32)
    for split in ([2, 0, 5, 1, 4], [0, 12, 0, 0, 0], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0]):
        s.copy_(dev_split(split))
        graph.replay()
        assert np.array_equal(out.double().cpu().numpy(), by_expert(x, split, lambda e, v: v @ b.values[e].T, n))
    s.copy_(dev_split([3, 3, 0, 3, 3]))
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gsa.grouped_gemv(xd, qb, s, n, recipe, out_dtype=torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out) and gsa.grouped_gemm_status(side) == 0
    frame = torch.full((16, n), 7.0, device="cuda")
    gsa.grouped_gemv(xd, qb, s, n, recipe, out=frame[2:14])
    assert torch.equal(frame[2:14], out) and bool((frame[:2] == 7).all()) and bool((frame[14:] == 7).all())


def test_bad_splits_and_no_rows():
    rng = np.random.default_rng(25)
    b, gated = Matrices(rng, [64, 64], 64, MX).dev(), Matrices(rng, [32] * 4, 64, MX).dev()
    x = torch.ones((6, 64), dtype=torch.bfloat16, device="cuda")
    for bad in ([3, 4], [-1, 3], [1 << 40, 0], [6, -(1 << 62)]):
        out = torch.full((6, 64), 5.0, device="cuda")
        gsa.grouped_gemv(x, b, dev_split(bad), 64, MX, out=out)
        assert gsa.grouped_gemm_status() == 1 and bool((out == 5).all())
        out = torch.full((6, 32), 5.0, device="cuda")
        gsa.grouped_glu_gemv(x, gated, dev_split(bad), 32, MX, b_groups=2, out=out)
        assert gsa.grouped_gemm_status() == 1 and bool((out == 5).all())
    assert gsa.grouped_gemv(x[:0], b, dev_split([0, 0]), 64, MX).shape == (0, 64)
    assert bool((gsa.grouped_gemv(x, b, dev_split([0, 0]), 64, MX) == 0).all()) and gsa.grouped_gemm_status() == 0


def test_python_refusals():
    rng = np.random.default_rng(26)
    b, s = Matrices(rng, [64, 64], 64, NV).dev(), dev_split([2, 2])
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: gsa.grouped_gemv(x.double(), b, s, 64, NV), lambda: gsa.grouped_gemv(x[0], b, s, 64, NV),
                 lambda: gsa.grouped_gemv(x.t(), b, s, 64, NV), lambda: gsa.grouped_gemv(x.cpu(), b, s, 64, NV),
                 lambda: gsa.grouped_gemv(x[:, :32].contiguous(), b, s, 64, NV), lambda: gsa.grouped_gemv(x, b, s, 65, NV),
                 lambda: gsa.grouped_gemv(x, b, None, 64, 2), lambda: gsa.grouped_gemv(x, {}, s, 64, NV),
                 lambda: gsa.grouped_gemv(x, b, s.int(), 64, NV), lambda: gsa.grouped_gemv(x, b, s[None], 64, NV),
                 lambda: gsa.grouped_gemv(x, b, s.cpu(), 64, NV), lambda: gsa.grouped_gemv(x, b, s, 64, NV, out_dtype=torch.float64),
                 lambda: gsa.grouped_gemv(x, b, s, 64, NV, out=torch.empty((4, 65), device="cuda")),
                 lambda: gsa.grouped_gemv(x, dict(b, amax_row=b["amax_row"][:1]), s, 64, NV),
                 lambda: gsa.grouped_glu_gemv(x, b, s, 32, NV), lambda: gsa.grouped_glu_gemv(x, b, s, 32, NV, b_groups=2),
                 lambda: gsa.grouped_glu_gemv(x, b, s, 32, NV, act="identity", b_groups=2),
                 lambda: gsa.grouped_glu_gemv(x, b, s, 32, NV, probs=torch.ones(3, device="cuda"), b_groups=2)):
        with pytest.raises(gsa.GsaError):
            call()
