"""The gated first projection and its gradient against their formulas in 64 bits.

Operands are codes and power-of-two scales for which every partial sum is exact in FP32 (as in the tests of the grouped
products), scaled so that the gate is a few units wide.  What is left is the activation's own error, bounded per element:
with u = 2^-24, E = e^-z is off by (4 + 3 |z|) u of itself (the rate -alpha log2 e, a product, the hardware's base-2
exponential within 2^-22), 1 + E by u, its reciprocal by 2u, E s by u: s and 1 - s by (8 + 3 |z|) u.  A product or sum adds u.  Padding of the scale tiles holds NaN, which no result may see."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, SPLITS, Matrices, dev_split

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

U = 2.0 ** -24
PARAMS = {"swiglu": (np.inf, 1.0, 0.0), "clamped_swiglu": (1.5, 1.702, 1.0)}
TYPES = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def gsa_params(act):
    limit, alpha, off = PARAMS[act]
    return gsa.act_params(act, limit=min(limit, 7.0), alpha=alpha, glu_linear_offset=off)


def shrink(m, recipe, k):
    """The same matrices in a unit that is a power of two, so that a product of two of them has entries of about 2."""
    bits = int(round(np.log2(12 * np.sqrt(k) / 2) / 2))
    if recipe == MX:
        m.scale = np.where(m.scale == 0xFF, m.scale, m.scale - bits).astype(np.uint8)
    else:
        m.amax = (m.amax * 2.0 ** -bits).astype(np.float32)
    m.values = [v * 2.0 ** -bits for v in m.values]
    return m


class Case:
    """Rows, weights (an expert's gate and linear rows as two groups, or as one), probs, dy, and the tail of rows."""

    def __init__(self, seed, recipe, split, n, k, groups, tail=0):
        rng = np.random.default_rng(seed)
        self.recipe, self.split, self.n, self.k, self.groups, self.rows = recipe, split, n, k, groups, sum(split)
        self.m = self.rows + tail
        self.a = shrink(Matrices(rng, split, k, recipe), recipe, k)
        self.b = shrink(Matrices(rng, [2 * n // groups] * (groups * len(split)), k, recipe), recipe, k)
        self.qa, self.qb, self.dev = self.a.dev(), self.b.dev(), dev_split(split)
        if tail:
            more = Matrices(rng, [tail], k, recipe).dev()["row_data"]
            self.qa["row_data"] = torch.cat((self.qa["row_data"][:self.a.data.size - 1], more))
        self.p = rng.uniform(-1, 1, self.m).astype(np.float32)
        self.probs = torch.from_numpy(self.p).cuda()
        self.dy_dev = torch.from_numpy(rng.standard_normal((self.m, n)).astype(np.float32)).cuda().to(torch.bfloat16)
        self.dy = self.dy_dev.double().cpu().numpy()
        g, u = [], []
        for e, x in enumerate(self.a.values):
            w = np.concatenate(self.b.values[e * groups:(e + 1) * groups])
            g.append(x @ w[:n].T)
            u.append(x @ w[n:].T)
        pad = [np.zeros((tail, n))]
        self.g, self.u = np.concatenate(g + pad), np.concatenate(u + pad)

    def args(self):
        return (self.qa, self.qb, self.dev, self.m, self.n, self.k, self.recipe)


def forward_ref(c, act, probs=True):
    """(y, the bound of its error before the last rounding)."""
    limit, alpha, off = PARAMS[act]
    a, b = np.minimum(c.g, limit), np.clip(c.u, -limit, limit) + off
    z = alpha * a
    s = 1 / (1 + np.exp(-z))
    y = a * s * b * (c.p[:, None].astype(np.float64) if probs else 1.0)
    rel = 16 + 3 * np.abs(z)   # z itself (clamped: a rounding of alpha a), s, the sum b, three products
    return y, rel * U * np.abs(y) + 4 * U * np.abs(a * s) * np.abs(off) + 2.0 ** -120


def gradient_ref(c, act, probs=True):
    limit, alpha, off = PARAMS[act]
    a, b = np.minimum(c.g, limit), np.clip(c.u, -limit, limit) + off
    z = alpha * a
    s = 1 / (1 + np.exp(-z))
    q = 1 / (1 + np.exp(z))
    t = c.dy * (c.p[:, None].astype(np.float64) if probs else 1.0)
    t[c.rows:] = 0.0   # rows that no expert has
    dg, du = t * b * (s + z * s * q) * (c.g <= limit), t * a * s * (np.abs(c.u) <= limit)
    rel = 2 * (16 + 3 * np.abs(z)) * U
    bg = rel * np.abs(t) * (np.abs(b) + np.abs(off)) * (s + np.abs(z) * s * q) + 2.0 ** -120
    bu = rel * np.abs(du) + 2.0 ** -120
    v = c.dy * a * s * b
    # a chain of 64 products and sums, then the partial sums
    bp = (np.abs(v) * (16 + 3 * np.abs(z) + 4 * np.abs(off) + 64 + 2 * -(-c.n // 128))).sum(1) * U + 2.0 ** -120
    return np.concatenate((dg, du), 1), np.concatenate((bg, bu), 1), v.sum(1), bp


def near(got, ref, bound, last):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= bound + last * (np.abs(ref) + bound))


SHAPES = [(1, 64, 2), (8, 128, 2), (100, 192, 2), (128, 256, 1), (257, 320, 2), (256, 1024, 1), (576, 576, 2), (130, 64, 2)]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("act", sorted(PARAMS))
@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("n,k,groups", SHAPES)
def test_forward_and_gradient(recipe, act, split, n, k, groups):
    tail = 3 if n % 2 else 200
    c = Case(n * 7 + k + len(split), recipe, split, n, k, groups, tail)
    more = {"act": act, "probs": c.probs, "params": gsa_params(act), "b_groups": groups}
    y, by = forward_ref(c, act)
    dx, bx, dp, bp = gradient_ref(c, act)
    for dtype, last in TYPES.items():
        out = torch.full((c.m, n), float("nan"), dtype=dtype, device="cuda")
        got = gsa.grouped_glu(*c.args(), **more, out=out)
        assert got is out
        near(got, y, by, last)
        outs = (torch.full((c.m, 2 * n), float("nan"), dtype=dtype, device="cuda"), torch.full((c.m,), float("nan"), device="cuda"))
        got = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more, out=outs)
        assert got[0] is outs[0] and got[1] is outs[1]
        near(got[0], dx, bx, last)
        near(got[1], dp, bp, U)
        for v in (out, *outs):
            assert bool((v[c.rows:] == 0).all())
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("rows", [20, 300])
def test_outputs_one_by_one(recipe, rows):
    """No probs, no dx, no dprobs: the same values as together, bit for bit; and each call twice the same."""
    c = Case(3, recipe, [rows, 0, rows], 136, 256, 2)
    y = gsa.grouped_glu(*c.args(), b_groups=2)
    ones = torch.ones(c.m, device="cuda")
    assert torch.equal(y, gsa.grouped_glu(*c.args(), b_groups=2, probs=ones))
    near(y, *forward_ref(c, "swiglu", False), 2.0 ** -8)
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2)
    only_x, none = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2, want_dprobs=False)
    none_x, only_p = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2, want_dx=False)
    assert none is None and none_x is None and torch.equal(dx, only_x) and torch.equal(dp, only_p)
    again = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2, probs=ones)
    assert torch.equal(dx, again[0]) and torch.equal(dp, again[1])


@pytest.mark.parametrize("recipe", [MX, NV])
def test_one_group_and_two_agree(recipe):
    """With n a multiple of 128 the scales lie alike; two groups bring a tensor scale each."""
    c = Case(4, recipe, [70, 300], 256, 320, 1)
    two = dict(c.qb, amax_row=c.qb["amax_row"].repeat_interleave(2))
    assert torch.equal(gsa.grouped_glu(*c.args()), gsa.grouped_glu(c.qa, two, *c.args()[2:], b_groups=2))
    if recipe == NV:   # gate and linear rows in units of their own: powers of two, so y changes with the linear one exactly
        far = dict(two, amax_row=two["amax_row"] * torch.tensor([1.0, 8.0] * 2, device="cuda"))
        assert torch.equal(8 * gsa.grouped_glu(*c.args()), gsa.grouped_glu(c.qa, far, *c.args()[2:], b_groups=2))


PAIRS = [(3e38, 1e-30), (1e-30, 3e38), (3e38, 1e-33), (1e-33, 1e30), (1e20, 1e-20)]


def test_units_far_apart():
    """NVFP4 units beyond FP32's range of products, with gate and linear rows of one group: g and u of ordinary size come
    out as the formulas say.  A sigmoid below 2^-126 is flushed to 0, which is 2^-126 |g u| of y.  1 / S of either side and its products add 4 units of 2^-23 to g and u, which y, its
    derivatives included, takes at most (4 + 2 |z|) times."""
    rng = np.random.default_rng(6)
    n, k, split = 128, 128, [40] * len(PAIRS)
    a, b = Matrices(rng, split, k, NV, [p[0] for p in PAIRS]), Matrices(rng, [2 * n] * len(PAIRS), k, NV, [p[1] for p in PAIRS])
    got = gsa.grouped_glu(a.dev(), b.dev(), dev_split(split), sum(split), n, k, NV, out_dtype=torch.float32).double().cpu().numpy()
    for e, (x, w) in enumerate(zip(a.values, b.values)):
        ux, uw = np.float64(a.amax[e]) / 2688.0, np.float64(b.amax[e]) / 2688.0
        h = (np.round(x / ux * 4) @ np.round(w / uw * 4).T) / 16 * ux * uw
        g, u = h[:, :n], h[:, n:]
        s = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
        ref = g * s * u
        bound = (16 + 3 * np.abs(g) + 8 * (4 + 2 * np.abs(g))) * U * np.abs(ref) + 2.0 ** -120 + 2.0 ** -125 * np.abs(g * u)
        assert np.all(np.abs(got[40 * e:40 * e + 40] - ref) <= bound), PAIRS[e]


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("rows", [50, 200])
def test_nan_stays_in_its_row_and_column(recipe, rows):
    """A NaN block scale of a row or of a weight row spoils that row and that column of that expert alone."""
    c = Case(8, recipe, [rows, rows], 150, 256, 2)
    nan = 0xFF if recipe == MX else 0x7F
    tiles = -(-(c.k // (32 if recipe == MX else 16)) // 4) * 512
    side = -(-c.n // 128) * tiles                                  # scale bytes of one group of weight rows
    c.qa["row_scale"][-(-rows // 128) * tiles + 16 * 5 + 2] = nan  # expert 1, row 5
    c.qb["row_scale"][3 * side + 16 * 7 + 4 * 1] = nan             # expert 1, linear row 39
    c.qb["row_scale"][2 * side + tiles + 16 * 3] = nan             # expert 1, gate row 131
    bad = np.zeros((c.m, c.n), bool)
    bad[rows + 5] = True
    bad[rows:, [39, 131]] = True
    more = {"act": "clamped_swiglu", "params": gsa_params("clamped_swiglu"), "b_groups": 2, "probs": c.probs}
    y = gsa.grouped_glu(*c.args(), **more, out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(y), bad)
    ref, by = forward_ref(c, "clamped_swiglu")
    assert np.all((np.abs(y - ref) <= by + U * np.abs(ref))[~bad])
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more, out_dtype=torch.float32)
    dx, dp = dx.cpu().numpy(), dp.cpu().numpy()
    ref, bx, _, _ = gradient_ref(c, "clamped_swiglu")
    fine = ~np.concatenate((bad, bad), 1)
    assert np.all((np.abs(dx - ref) <= bx + U * np.abs(ref))[fine])
    assert np.array_equal(np.isnan(dp), bad.any(1))
    assert np.isnan(dx[rows + 5]).all()


def test_values_at_the_ends_of_the_range():
    """Pre-activations of 2^+-60 and zeros: the gate's sigmoid is 0, 1/2 or 1 and nothing becomes NaN."""
    n, k = 128, 64
    code = np.array([0x38, 0xB8], np.uint8)                        # E4M3 1 and -1
    scales = np.array([127 + 60, 127 - 60, 127, 0], np.uint8)      # rows of 2^60, 2^-60, 1, 2^-127
    data = np.zeros((8, k), np.uint8)
    tiles = np.zeros(512, np.uint8)
    for r in range(8):
        data[r, 0] = code[r // 4]
        tiles[16 * r:16 * r + 2] = scales[r % 4]
    w, wt = np.zeros((2 * n, k), np.uint8), np.full(1024, 127, np.uint8)
    w[:, 0] = 0x38
    q = {"row_data": torch.from_numpy(data).cuda(), "row_scale": torch.from_numpy(tiles).cuda()}
    qw = {"row_data": torch.from_numpy(w).cuda(), "row_scale": torch.from_numpy(wt).cuda()}
    x = np.array([2.0 ** 60, 2.0 ** -60, 1.0, 2.0 ** -127, -2.0 ** 60, -2.0 ** -60, -1.0, -2.0 ** -127])
    y = gsa.grouped_glu(q, qw, dev_split([8]), 8, n, k, MX, out_dtype=torch.float32).double().cpu().numpy()
    s = 1 / (1 + np.exp(-np.clip(x, -700, 700)))
    ref = x * s * x
    assert np.all(np.abs(y - ref[:, None]) <= 20 * U * np.abs(ref)[:, None] + 2.0 ** -120)
    dy = torch.ones((8, n), dtype=torch.bfloat16, device="cuda")
    dx, dp = gsa.grouped_glu_bwd(dy, q, qw, dev_split([8]), 8, n, k, MX, out_dtype=torch.float32)
    c = 1 / (1 + np.exp(np.clip(x, -700, 700)))
    dg, du = x * (s + x * s * c), x * s
    for got, want in ((dx[:, :n], dg), (dx[:, n:], du)):
        assert np.all(np.abs(got.double().cpu().numpy() - want[:, None]) <= 50 * U * np.abs(want)[:, None] + 2.0 ** -120)
    assert np.all(np.abs(dp.double().cpu().numpy() - n * ref) <= (20 + 64 + 2) * U * np.abs(n * ref) + 2.0 ** -113)


def test_gradient_against_differences():
    """Central differences of sum(dy y) along the units of two experts' gate and linear sides and of probs: scaling a side's
    tensor scale by 1 + h moves all of its pre-activations by h of themselves, so the derivative is the sum of x dx over
    the side.  Errors: h^2 |third derivative| and 2^-23 of the sums' magnitude over h."""
    c = Case(12, NV, [33, 200], 136, 192, 2)
    act = {"act": "clamped_swiglu", "params": gsa.act_params("clamped_swiglu", limit=50.0, alpha=1.25, glu_linear_offset=0.5),
           "b_groups": 2, "out_dtype": torch.float32}
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), probs=c.probs, **act)
    dx, dy, h = dx.double().cpu().numpy(), c.dy, 2.0 ** -7

    def value(amax, probs):
        y = gsa.grouped_glu(c.qa, dict(c.qb, amax_row=amax), *c.args()[2:], probs=probs, **act)
        return y.double().cpu().numpy() * dy

    rows = [slice(0, 33), slice(33, 233)]
    for e in range(2):
        for side, pre in ((0, c.g), (1, c.u)):
            step = torch.ones(4, device="cuda")
            step[2 * e + side] = 1 + h
            down = torch.ones(4, device="cuda")
            down[2 * e + side] = 1 - h
            up, low = value(c.qb["amax_row"] * step, c.probs), value(c.qb["amax_row"] * down, c.probs)
            diff = (up - low)[rows[e]].sum() / (2 * h)
            own = (dx[rows[e], side * c.n:(side + 1) * c.n] * pre[rows[e]]).sum()
            mass = np.abs(dx[rows[e], side * c.n:(side + 1) * c.n] * pre[rows[e]])
            # third derivative of x s(z) b along ln x: within 8 (1 + |z|)^3 of the value; 1 +- h is exact in FP32
            third = (8 * (1 + 1.25 * np.abs(c.g[rows[e]])) ** 3 * np.abs(up[rows[e]])).sum() if side == 0 else 0.0
            assert abs(diff - own) <= h * h / 6 * third + 2.0 ** -21 / h * np.abs(up[rows[e]]).sum() + 2.0 ** -20 * mass.sum()
    ones = torch.ones(c.m, device="cuda")
    v = value(c.qb["amax_row"], ones).sum(1)
    bound = (64 + 60) * U * np.abs(value(c.qb["amax_row"], ones)).sum(1) + 2.0 ** -100
    assert np.all(np.abs(dp.double().cpu().numpy() - v) <= bound)


@pytest.mark.parametrize("recipe", [MX, NV])
def test_graph_stream_and_determinism(recipe):
    """Captured and replayed with another split in place, on another stream, and the same bits each time."""
    splits = [[300, 17, 0, 64], [1, 200, 180, 0]]
    cs = [Case(13 + i, recipe, s, 136, 192, 2) for i, s in enumerate(splits)]
    size = max(c.qa["row_data"].numel() for c in cs), max(c.qa["row_scale"].numel() for c in cs)
    qa = {"row_data": torch.zeros(size[0], dtype=torch.uint8, device="cuda"),
          "row_scale": torch.zeros(size[1], dtype=torch.uint8, device="cuda"), "amax_row": cs[0].qa["amax_row"].clone()}
    qb, split, dy = {k: v.clone() for k, v in cs[0].qb.items()}, cs[0].dev.clone(), torch.zeros((381, 136), dtype=torch.bfloat16, device="cuda")
    probs = torch.zeros(381, device="cuda")

    def call(stream=None):
        y = gsa.grouped_glu(qa, qb, split, 381, 136, 192, recipe, probs=probs, b_groups=2, out_dtype=torch.float32, stream=stream)
        return (y, *gsa.grouped_glu_bwd(dy, qa, qb, split, 381, 136, 192, recipe, probs=probs, b_groups=2, stream=stream))

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
        dy[:c.m].copy_(c.dy_dev)
        probs[:c.m].copy_(c.probs)
        graph.replay()
        near(outs[0][:c.m], *forward_ref(c, "swiglu"), U)
        dx, bx, dp, bp = gradient_ref(c, "swiglu")
        near(outs[1][:c.m], dx, bx, 2.0 ** -8)
        near(outs[2][:c.m], dp, bp, U)
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(u, v) for u, v in zip(got, outs))
    assert gsa.grouped_gemm_status() == 0


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("rows", [30, 300])
def test_bad_splits_write_nothing(recipe, rows):
    c = Case(15, recipe, [rows, rows], 128, 64, 1)
    for bad in ([rows, rows + 1], [-1, rows], [1 << 40, 0], [2 * rows, -(1 << 62)]):
        y, dx = torch.full((c.m, 128), 5.0, device="cuda"), torch.full((c.m, 256), 5.0, device="cuda")
        dp = torch.full((c.m,), 5.0, device="cuda")
        args = (c.qa, c.qb, dev_split(bad), *c.args()[3:])
        gsa.grouped_glu(*args, out=y)
        assert gsa.grouped_gemm_status() == 1
        gsa.grouped_glu_bwd(c.dy_dev, *args, out=(dx, dp))
        assert gsa.grouped_gemm_status() == 1 and gsa.grouped_gemm_status() == 0
        assert bool((y == 5).all()) and bool((dx == 5).all()) and bool((dp == 5).all())


def test_no_rows_and_no_live_rows():
    c = Case(16, MX, [0, 0], 128, 64, 1, tail=5)
    q0 = dict(c.qa, row_data=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    y = gsa.grouped_glu(*c.args())
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args())
    assert bool((y == 0).all()) and bool((dx == 0).all()) and bool((dp == 0).all()) and y.shape == (5, 128)
    args = (q0, c.qb, c.dev, 0, 128, 64, MX)
    assert gsa.grouped_glu(*args).shape == (0, 128)
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev[:0], *args)
    assert dx.shape == (0, 256) and dp.shape == (0,) and gsa.grouped_gemm_status() == 0


def test_python_refusals():
    c = Case(17, NV, [4, 4], 128, 64, 1)
    a, b, s, m, n, k, r = c.args()
    odd = Case(18, NV, [4, 4], 64, 64, 2)
    for call in (lambda: gsa.grouped_glu(a, b, s, m, n, k, r, act="srelu"), lambda: gsa.grouped_glu(a, b, s, m, n, k, r, act="nothing"),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, b_groups=3),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, b_groups=2),                  # amax of two groups missing
                 lambda: gsa.grouped_glu(*odd.args(), b_groups=1),                          # scales inside a tile
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, probs=c.probs[:3]),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, probs=c.probs.double()),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, act="clamped_swiglu", params=gsa.act_params("clamped_swiglu", limit=0.0)),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, act="clamped_swiglu", params=gsa.act_params("clamped_swiglu", alpha=float("inf"))),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, out_dtype=torch.float16),
                 lambda: gsa.grouped_glu(a, b, s, m, n, k, r, out=torch.empty((m, 2 * n), device="cuda")),
                 lambda: gsa.grouped_glu(a, b, s, m, 2 * n, k, r), lambda: gsa.grouped_glu(a, b, s.int(), m, n, k, r),
                 lambda: gsa.grouped_glu(a, b, s, m + 1, n, k, r), lambda: gsa.grouped_glu({}, b, s, m, n, k, r),
                 lambda: gsa.grouped_glu_bwd(c.dy_dev.float(), a, b, s, m, n, k, r),
                 lambda: gsa.grouped_glu_bwd(c.dy_dev[:, :64], a, b, s, m, n, k, r),
                 lambda: gsa.grouped_glu_bwd(c.dy_dev, a, b, s, m, n, k, r, want_dx=False, want_dprobs=False),
                 lambda: gsa.grouped_glu_bwd(c.dy_dev, a, b, s, m, n, k, r, out=(None, torch.empty(m + 1, device="cuda")))):
        with pytest.raises(gsa.GsaError):
            call()


@pytest.mark.parametrize("recipe", [MX, NV])
def test_long_sums(recipe):
    """Rows of one sign over 65536 columns of k: a piece of the gradient's sums is 64 steps of 32 bytes, each cutting off less
    than 2^-23 of the running sum: (64 + 1) / 2 units and one for each of the pieces (32 or 64, half a unit each), so g and
    u are within 65 units of 2^-23 of themselves.  The forward's FP32 result has the same pieces, and y, dx and dp are
    products of at most two of them (the gate far to the right: its sigmoid is 1)."""
    from test_gpu_grouped_gemm_long import positive
    rng = np.random.default_rng(5)
    k, n, rows = 65536, 128, 40
    da, sa, va = positive(rng, rows, k, recipe)
    db, sb, vb = positive(rng, 2 * n, k, recipe)
    amax = torch.full((1,), 2688.0, device="cuda")
    qa, qb = ({"row_data": torch.from_numpy(d).cuda(), "row_scale": torch.from_numpy(s).cuda(), "amax_row": amax} for d, s in ((da, sa), (db, sb)))
    h = va @ vb.T
    g, u = h[:, :n], h[:, n:]
    assert g.min() > 100
    y = gsa.grouped_glu(qa, qb, dev_split([rows]), rows, n, k, recipe, out_dtype=torch.float32).double().cpu().numpy()
    assert np.max(np.abs(y / (g * u) - 1)) <= 2 * 66 * 2.0 ** -23
    dy = torch.ones((rows, n), dtype=torch.bfloat16, device="cuda")
    dx, dp = gsa.grouped_glu_bwd(dy, qa, qb, dev_split([rows]), rows, n, k, recipe, out_dtype=torch.float32)
    dx, dp = dx.double().cpu().numpy(), dp.double().cpu().numpy()
    assert np.max(np.abs(dx[:, :n] / u - 1)) <= 66 * 2.0 ** -23 and np.max(np.abs(dx[:, n:] / g - 1)) <= 66 * 2.0 ** -23
    assert np.max(np.abs(dp / (g * u).sum(1) - 1)) <= (2 * 66 + 33 + 2) * 2.0 ** -23
