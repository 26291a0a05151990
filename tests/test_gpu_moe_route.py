"""Tokens into expert order and back (gsa_moe_*) against plain NumPy forms in
64 bits: the sort plan exactly, row moves bit for bit, and sums within bounds
that follow from the arithmetic: FP32 accumulation of m terms is off by at most
m 2^-24 sum |terms| (one rounding per fused multiply-add), and the result's own
rounding adds half a unit of its type, 2^-9 (BF16), 2^-12 (FP16) or 2^-25 (FP32)
of its size doubled to cover the double rounding."""
import numpy as np
import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}   # subnormal steps
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make_idx(rng, tokens, topk, experts, drop=0.0, dtype=np.int64):
    idx = rng.integers(0, experts, size=(tokens, topk))
    if drop:
        gone = rng.random((tokens, topk)) < drop
        idx = np.where(gone, rng.choice([-1, experts, experts + 5, -7], size=idx.shape), idx)
        if tokens:
            idx[tokens // 2] = -1
    return idx.astype(dtype)


def plan(idx, experts):
    key = np.where((idx < 0) | (idx >= experts), experts, idx).reshape(-1).astype(np.int64)
    order = np.argsort(key, kind="stable")
    row = np.empty(key.size, np.int64)
    row[order] = np.arange(key.size)
    row = np.where(key == experts, ~row, row).reshape(idx.shape)
    return row.astype(np.int32), np.bincount(key, minlength=experts + 1)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def normal(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def check_sum(got, ref, mass, terms, dtype):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= terms * 2.0 ** -24 * mass + ROUND[dtype] * np.abs(ref) + TINY[dtype])


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("tokens,topk,experts", [(0, 3, 4), (1, 1, 1), (1, 8, 128), (16, 8, 128), (33, 2, 3), (1000, 7, 256),
                                                 (1024, 8, 64), (1025, 8, 64), (2731, 3, 7), (20011, 5, 256),
                                                 (262147, 4, 31)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort_plan(tokens, topk, experts, drop, dtype):
    rng = np.random.default_rng(tokens + topk * 7 + experts)
    idx = make_idx(rng, tokens, topk, experts, drop, dtype)
    row, split = gsa.moe_sort(dev(idx), experts)
    ref_row, ref_split = plan(idx, experts)
    assert np.array_equal(row.cpu().numpy(), ref_row)
    assert np.array_equal(split.cpu().numpy(), ref_split)


@pytest.mark.parametrize("how", ["one expert", "all dropped", "sorted", "reversed"])
def test_sort_plan_skewed(how):
    tokens, topk, experts = 6007, 2, 40
    idx = {"one expert": np.full((tokens, topk), 17), "all dropped": np.full((tokens, topk), -1),
           "sorted": np.arange(tokens * topk).reshape(tokens, topk) * experts // (tokens * topk),
           "reversed": experts - 1 - np.arange(tokens * topk).reshape(tokens, topk) * experts // (tokens * topk)}[how]
    row, split = gsa.moe_sort(dev(idx.astype(np.int64)), experts)
    ref_row, ref_split = plan(idx, experts)
    assert np.array_equal(row.cpu().numpy(), ref_row) and np.array_equal(split.cpu().numpy(), ref_split)


# widths: vector multiples, 8-, 4- and 2-byte rows, one element, beyond one block's columns
SHAPES = [(1, 1, 4, 64), (1, 8, 128, 4096), (5, 3, 7, 1), (37, 2, 5, 1111), (37, 9, 16, 1110), (64, 8, 16, 1108),
          (130, 4, 8, 2048), (3, 17, 33, 300), (19, 6, 256, 8200), (3000, 2, 9, 72), (700, 5, 3, 66)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,hidden", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_permute_and_gradient(tokens, topk, experts, hidden, drop, dtype):
    rng = np.random.default_rng(hidden + tokens)
    row, _ = plan(make_idx(rng, tokens, topk, experts, drop), experts)
    n, live, at = tokens * topk, row >= 0, np.maximum(row, ~row)
    x, probs = normal(rng, (tokens, hidden), dtype), normal(rng, (tokens, topk), torch.float32)
    xs, ps = gsa.moe_permute(x, dev(row), probs)
    ref, refp = np.zeros((n, hidden)), np.zeros(n)
    ref[at[live]] = f64(x)[np.nonzero(live)[0]]
    refp[at[live]] = f64(probs)[live]
    assert np.array_equal(f64(xs), ref) and np.array_equal(f64(ps), refp)
    assert torch.equal(gsa.moe_permute(x, dev(row)), xs)

    dxs, dps = normal(rng, (n, hidden), dtype), normal(rng, (n,), torch.float32)
    gone = dev(at[~live].astype(np.int64))
    dxs[gone], dps[gone] = float("nan"), float("nan")   # never read
    dx, dprobs = gsa.moe_permute_bwd(dxs, dev(row), dps)
    v = np.where(live[:, :, None], f64(dxs)[at], 0.0)
    check_sum(dx, v.sum(1), np.abs(v).sum(1), topk, dtype)
    assert np.array_equal(f64(dprobs), np.where(live, f64(dps)[at], 0.0))
    assert torch.equal(gsa.moe_permute_bwd(dxs, dev(row)), dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,hidden", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("weighted", [True, False])
def test_unpermute_and_gradient(tokens, topk, experts, hidden, drop, dtype, weighted):
    rng = np.random.default_rng(hidden * 3 + tokens)
    row, _ = plan(make_idx(rng, tokens, topk, experts, drop), experts)
    n, live, at = tokens * topk, row >= 0, np.maximum(row, ~row)
    ys = normal(rng, (n, hidden), dtype)
    ys[dev(at[~live].astype(np.int64))] = float("nan")   # never read
    w = normal(rng, (tokens, topk), torch.float32) if weighted else None
    wf = f64(w) if weighted else np.ones((tokens, topk))
    out = gsa.moe_unpermute(ys, dev(row), w)
    y = np.where(live[:, :, None], f64(ys)[at], 0.0)
    terms = wf[:, :, None] * y
    check_sum(out, terms.sum(1), np.abs(terms).sum(1), topk, dtype)

    dout = normal(rng, (tokens, hidden), dtype)
    dys, dw = gsa.moe_unpermute_bwd(dout, ys, dev(row), w)
    ref = np.zeros((n, hidden))
    ref[at[live]] = (wf[:, :, None] * f64(dout)[:, None, :])[live]
    check_sum(dys, ref, np.abs(ref), 1, dtype)
    terms = y * f64(dout)[:, None, :]
    check_sum(dw, np.where(live, terms.sum(2), 0.0), np.abs(terms).sum(2), hidden, torch.float32)
    only, none = gsa.moe_unpermute_bwd(dout, None, dev(row), w)
    assert none is None and torch.equal(only, dys)
    none, only = gsa.moe_unpermute_bwd(dout, ys, dev(row), w, want_dys=False)
    assert none is None and torch.equal(only, dw)


def test_gradients_against_differences():
    """unpermute is linear in the rows and in the weights, so central
    differences with step 1 are exact but for rounding: both sides sum FP32
    values whose errors are bounded as above, here summed over the outputs."""
    rng = np.random.default_rng(5)
    tokens, topk, experts, hidden = 23, 4, 6, 96
    row, _ = plan(make_idx(rng, tokens, topk, experts, 0.2), experts)
    n, dt = tokens * topk, torch.float32
    ys, dout = normal(rng, (n, hidden), dt), normal(rng, (tokens, hidden), dt)
    w, r = normal(rng, (tokens, topk), dt), dev(row)
    dys, dw = gsa.moe_unpermute_bwd(dout, ys, r, w)
    dx = gsa.moe_permute_bwd(ys, r)

    def loss(out):
        return float(np.sum(f64(out) * f64(dout)))

    vy, vw, vx = normal(rng, (n, hidden), dt), normal(rng, (tokens, topk), dt), normal(rng, (tokens, hidden), dt)
    # |loss| terms are at most (|w|+|vw|)(|y|+|vy|)|dout| <= 6.5^3 each, topk of them per output element
    bound = (topk + 3) * 2.0 ** -24 * 6.5 ** 3 * topk * tokens * hidden
    by_ys = (loss(gsa.moe_unpermute(ys + vy, r, w)) - loss(gsa.moe_unpermute(ys - vy, r, w))) / 2
    assert abs(by_ys - float(np.sum(f64(dys) * f64(vy)))) <= bound
    by_w = (loss(gsa.moe_unpermute(ys, r, w + vw)) - loss(gsa.moe_unpermute(ys, r, w - vw))) / 2
    assert abs(by_w - float(np.sum(f64(dw) * f64(vw)))) <= bound
    by_x = (float(np.sum(f64(gsa.moe_permute(dout + vx, r)) * f64(ys))) -
            float(np.sum(f64(gsa.moe_permute(dout - vx, r)) * f64(ys)))) / 2
    assert abs(by_x - float(np.sum(f64(dx) * f64(vx)))) <= bound


def test_special_values_and_foreign_plans():
    """Infinities and NaN travel with their rows only; a plan entry out of range is skipped."""
    row = dev(np.array([[0, 2], [1, 3], [-5, -6]], np.int32))
    ys = torch.ones((6, 64), device="cuda")
    ys[0], ys[2] = float("inf"), float("-inf")
    ys[3, 5] = float("nan")
    ys[4:] = float("nan")
    out = gsa.moe_unpermute(ys, row)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[1, 5])) and float(out[1, 4]) == 2.0
    assert bool((out[2] == 0).all())
    far = dev(np.array([[0, 1000], [-1000, 1], [2 ** 31 - 1, -2 ** 31]], np.int32))
    x = torch.ones((3, 64), device="cuda")
    xs, ps = gsa.moe_permute(x, far, torch.ones((3, 2), device="cuda"),
                             out=(torch.zeros((6, 64), device="cuda"), torch.zeros(6, device="cuda")))
    assert float(xs.sum()) == 128.0 and float(ps.sum()) == 2.0
    assert torch.equal(gsa.moe_unpermute(torch.ones((6, 64), device="cuda"), far)[:, 0].cpu(),
                       torch.tensor([1.0, 1.0, 0.0]))
    dys, dw = gsa.moe_unpermute_bwd(x, torch.ones((6, 64), device="cuda"), far,
                                    out=(torch.zeros((6, 64), device="cuda"), torch.empty((3, 2), device="cuda")))
    assert float(dys.sum()) == 128.0 and dw.cpu().tolist() == [[64.0, 0.0], [0.0, 64.0], [0.0, 0.0]]


def test_more_than_2_31_bytes():
    """Row offsets pass 32 bits: 70000 x 8 rows of 4096 BF16 (4.6 GB)."""
    tokens, topk, hidden, experts = 70000, 8, 4096, 11
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    idx = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda")
    row, split = gsa.moe_sort(idx, experts)
    x = torch.randn((tokens, hidden), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    xs = gsa.moe_permute(x, row)
    assert bool((xs[row.long().reshape(-1)].view(tokens, topk, hidden) == x[:, None, :]).all())
    out = gsa.moe_unpermute(xs, row)
    assert torch.equal(out, (x.float() * 8).to(torch.bfloat16))


def test_stream_and_graph():
    """Calls on a stream of their own, and a captured chain replayed on new inputs."""
    rng = np.random.default_rng(9)
    tokens, topk, experts, hidden = 96, 4, 12, 256
    s = torch.cuda.Stream()
    idx = dev(make_idx(rng, tokens, topk, experts, 0.1))
    x, w = normal(rng, (tokens, hidden), torch.bfloat16), normal(rng, (tokens, topk), torch.float32)
    s.wait_stream(torch.cuda.current_stream())
    row, split = gsa.moe_sort(idx, experts, stream=s)
    xs, ps = gsa.moe_permute(x, row, w, stream=s)
    out = gsa.moe_unpermute(xs, row, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    row2, _ = gsa.moe_sort(idx, experts)
    assert torch.equal(row, row2) and torch.equal(out, gsa.moe_unpermute(gsa.moe_permute(x, row2), row2, w))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        row, split = gsa.moe_sort(idx, experts)
        xs, ps = gsa.moe_permute(x, row, w)
        out = gsa.moe_unpermute(xs, row, w)
    idx.copy_(dev(make_idx(rng, tokens, topk, experts, 0.3)))
    x.copy_(normal(rng, (tokens, hidden), torch.bfloat16))
    graph.replay()
    row2, split2 = gsa.moe_sort(idx, experts)
    xs2, ps2 = gsa.moe_permute(x, row2, w)
    assert torch.equal(row, row2) and torch.equal(split, split2) and torch.equal(xs, xs2) and torch.equal(ps, ps2)
    assert torch.equal(out, gsa.moe_unpermute(xs2, row2, w))


def test_python_refusals():
    x = torch.zeros((4, 64), device="cuda")
    row = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for call in (lambda: gsa.moe_sort(torch.zeros(4, dtype=torch.int64, device="cuda"), 3),
                 lambda: gsa.moe_sort(torch.zeros((4, 2), device="cuda"), 3),
                 lambda: gsa.moe_sort(torch.zeros((4, 2), dtype=torch.int64), 3),
                 lambda: gsa.moe_sort(torch.zeros((4, 2), dtype=torch.int64, device="cuda"), 0),
                 lambda: gsa.moe_sort(torch.zeros((4, 2), dtype=torch.int64, device="cuda"), 257),
                 lambda: gsa.moe_permute(x[:3], row), lambda: gsa.moe_permute(x.double(), row),
                 lambda: gsa.moe_permute(x.t()[:4], row), lambda: gsa.moe_permute(x, row.long()),
                 lambda: gsa.moe_permute(x, row, torch.zeros((4, 3), device="cuda")),
                 lambda: gsa.moe_unpermute(x, row), lambda: gsa.moe_permute_bwd(x, row),
                 lambda: gsa.moe_unpermute(torch.zeros((8, 64), device="cuda"), row, torch.zeros(8, device="cuda")),
                 lambda: gsa.moe_unpermute(torch.zeros(8 * 64 + 1, device="cuda")[1:].view(8, 64), row),
                 lambda: gsa.moe_unpermute_bwd(x, torch.zeros((8, 32), device="cuda"), row)):
        with pytest.raises(gsa.GsaError):
            call()
