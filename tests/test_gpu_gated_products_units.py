"""Gated projections of NVFP4 operands whose two units (1 / S of either side) multiply to what FP32 does not hold: past its largest
value, below its smallest normal one, infinite.

A sum of codes and block scales is exact here.  Either unit is two divisions (one rounding each) and the two multiplications by
them one each: 6 roundings, so a pre-activation is within 6 U of itself, U = 2^-24, and half a subnormal step for each of
the multiplications where they end there.  With z = alpha g, s its sigmoid and q = 1 - s: g s moves by 1 + |z| q of g's share,
s + z s q by |z| s q (2 + |z|) times it.  The activation itself: e^-z is off by (4 + 3 |z|) U of itself (test_gpu_grouped_glu),
of which s takes q and q takes s; a sigmoid below 2^-126 is flushed."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import NV, Matrices, dev_split

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

U, STEP = 2.0 ** -24, 2.0 ** -149
PARAMS = {"swiglu": (np.inf, 1.0, 0.0), "clamped_swiglu": (1.5, 1.702, 1.0)}
K = 128


def unit(amax):
    """1 / S as a real number: what the operands' values are relative to."""
    return np.where(np.asarray(amax) > 0, np.float64(amax) / 2688.0, 1.0)


def least(m):
    """The same matrices with block scales of 2^-9 to 2^-7, the least that E4M3 has: sums are 2^-16 times as large."""
    power = (m.scale.astype(np.int64) >> 3) - 7                    # -1, 0 or 1
    m.scale = np.where(m.scale == 0x7F, m.scale, 1 << (power + 1)).astype(np.uint8)
    m.values = [v * 2.0 ** -8 for v in m.values]
    return m


def most(m):
    """Block scales of 2^6 to 2^8."""
    m.scale = np.where(m.scale == 0x7F, m.scale, m.scale + (7 << 3)).astype(np.uint8)
    m.values = [v * 128 for v in m.values]
    return m


class Case:
    """Experts with units of their own for rows, gate and linear rows."""

    def __init__(self, seed, rows, n, amax, sums, zero=False):
        rng = np.random.default_rng(seed)
        e = len(amax)
        self.split, self.n = [rows] * e, n
        self.m = rows * e
        of_a, of_gate, of_linear = (np.array(v, np.float32) for v in zip(*amax))
        self.a, self.b = sums(Matrices(rng, self.split, K, NV)), sums(Matrices(rng, [n] * (2 * e), K, NV))
        if zero:   # what the quantizer makes of an expert with an infinite value: S = 0
            self.a.data[:] = 0
            self.a.values = [0 * v for v in self.a.values]
        self.a.amax, self.b.amax = of_a, np.stack((of_gate, of_linear), 1).reshape(-1)
        self.qa, self.qb, self.dev = self.a.dev(), self.b.dev(), dev_split(self.split)
        self.dy_dev = torch.from_numpy(rng.standard_normal((self.m, n)).astype(np.float32)).cuda().to(torch.bfloat16)
        self.dy = self.dy_dev.double().cpu().numpy()
        ua, ug, ul = unit(of_a), unit(of_gate), unit(of_linear)
        with np.errstate(invalid="ignore"):
            side = [np.concatenate([x @ self.b.values[2 * i + j].T * ua[i] * u[i] for i, x in enumerate(self.a.values)])
                    for j, u in ((0, ug), (1, ul))]
        self.g, self.u = side

    def args(self):
        return self.qa, self.qb, self.dev, self.m, self.n, K, NV


def close(got, ref, bound):
    got = got.double().cpu().numpy()
    assert np.isfinite(ref).all() and np.max(np.abs(ref)) < 3e38
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


def check(c, act):
    limit, alpha, off = PARAMS[act]
    a, b = np.minimum(c.g, limit), np.clip(c.u, -limit, limit) + off
    z = alpha * a
    s, q = 1 / (1 + np.exp(-np.clip(z, -700, 700))), 1 / (1 + np.exp(np.clip(z, -700, 700)))
    az, w = np.abs(z), np.abs(z) * q
    more = {"act": act, "b_groups": 2, "out_dtype": torch.float32,
            "params": gsa.act_params(act, limit=min(limit, 7.0), alpha=alpha, glu_linear_offset=off)}
    tiny, flush = 8 * STEP, 2.0 ** -125   # of g, of u and of results that are subnormal; of a sigmoid
    y = a * s * b
    by = (16 + 3 * w + 6 * (2 + w)) * U * np.abs(y) + (4 + 6) * U * np.abs(a * s) * abs(off) + tiny * (1 + np.abs(a) + np.abs(b)) + flush * np.abs(a * b)
    close(gsa.grouped_glu(*c.args(), **more), y, by)
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), **more)
    dg, du = c.dy * b * (s + z * s * q) * (c.g <= limit), c.dy * a * s * (np.abs(c.u) <= limit)
    shape, bend = s + az * s * q, az * s * q * (2 + az)
    bg = U * np.abs(c.dy) * (np.abs(b) + abs(off)) * ((32 + 6 + 6) * shape + (6 + 6) * bend + 6 * w * s)
    bg += (tiny * (1 + np.abs(b)) + flush * np.abs(b) * (1 + w)) * np.abs(c.dy) + tiny
    bu = (32 + 6 * w + 6 * (1 + w)) * U * np.abs(du) + (tiny + flush * np.abs(a)) * np.abs(c.dy) + tiny
    close(dx[:, :c.n], dg, bg)
    close(dx[:, c.n:], du, bu)
    v = c.dy * y
    bp = (np.abs(c.dy) * by + (64 + 2 * -(-c.n // 128)) * U * np.abs(v) + STEP).sum(1)
    close(dp, v.sum(1), bp)
    assert gsa.grouped_gemm_status() == 0


def pairs(rows, n, e):
    """Whether blocks of a cluster take the call (test_gpu_gated_products_many_rows)."""
    return rows >= 128 and rows * e // 256 * -(-n // 128) >= 76


SIZES = [(40, 100, False), (700, 640, True)]

# sums of 2^-20 to 2^-6: units past 2^128 leave results in range
PAST = [(2688 * 2.0 ** 66, 2688 * 2.0 ** -58, 2688 * 2.0 ** 63), (2688 * 2.0 ** 20, 2688 * 2.0 ** 110, 2688 * 2.0 ** -112),
        (2688 * 2.0 ** 64, 2688 * 2.0 ** -56, 2688 * 2.0 ** 64), (2688 * 2.0 ** 112, 2688 * 2.0 ** -104, 2688 * 2.0 ** 17),
        (2688 * 2.0 ** 100, 2688 * 2.0 ** -92, 2688 * 2.0 ** 30), (2.5e38, 2688 * 2.0 ** -108, 1.6e7)]


@pytest.mark.parametrize("rows,n,pair", SIZES)
def test_units_past_the_largest_value(rows, n, pair):
    assert pairs(rows, n, len(PAST)) == pair
    check(Case(1, rows, n, PAST, least), "swiglu")


# sums of about 2^21: the units' product is subnormal, the pre-activations are not
BELOW = [(3e-16, 1e-16, 1.0), (1e-18, 2e-17, 1e-18), (2688 * 2.0 ** -66, 2688 * 2.0 ** -66, 2688 * 2.0 ** 60), (1e-33, 2e-2, 3.0),
         (3e-2, 1e-33, 1e-33), (3e3 * 2.0 ** -100, 3e3 * 2.0 ** -38, 1.0)]


@pytest.mark.parametrize("act", sorted(PARAMS))
@pytest.mark.parametrize("rows,n,pair", SIZES)
def test_units_below_the_smallest(act, rows, n, pair):
    """The clamped activation's offset carries a gate this small into y: g / 2 to FP32's precision."""
    assert pairs(rows, n, len(BELOW)) == pair
    check(Case(2, rows, n, BELOW, most), act)


@pytest.mark.parametrize("rows,n,pair", SIZES)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_infinite_units_show(rows, n, pair, which):
    """An infinite value makes S 0 and its expert's codes and sums with it: 0 times an infinite unit is NaN, in the gated product
    as in the plain one, and in that expert's results alone."""
    amax = [[2688.0 / 16] * 3 for _ in range(6)]
    amax[2][which] = np.inf
    c = Case(3, rows, n, amax, lambda m: m, zero=True)
    assert pairs(rows, n, 6) == pair
    hit = slice(2 * rows, 3 * rows)
    y = gsa.grouped_glu(*c.args(), b_groups=2)
    dx, dp = gsa.grouped_glu_bwd(c.dy_dev, *c.args(), b_groups=2)
    for t in (y, dx[:, :n] if which != 1 else dx[:, n:], dp[:, None]):
        nan = torch.isnan(t)
        assert bool(nan[hit].all()) and int(nan.sum()) == nan[hit].numel()
    plain = gsa.grouped_gemm(c.qa, dict(c.qb, amax_row=c.qb["amax_row"].view(-1, 2)[:, min(which, 2) // 2].contiguous()), c.dev, c.m, n, K, NV)
    assert bool(torch.isnan(plain[hit]).all())
    assert gsa.grouped_gemm_status() == 0
