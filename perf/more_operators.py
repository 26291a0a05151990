"""Workloads of the gated expert projections and of the products for single tokens.

Four operators on the experts' block-scaled (MXFP8 / NVFP4) weights:

* ``glu``       -- both halves of the first projection, the gated activation and
  the router's scale in one product: quantized rows, ragged over the experts.
* ``glu_grad``  -- its gradient: the pre-activations' gradient and the router
  scale's, with the pre-activations recomputed from the quantized rows.
* ``gemv``      -- a few unquantized rows an expert against its quantized weights
  (decoding).
* ``glu_gemv``  -- the gated first projection of such rows.

``own`` selects the framework's kernels; otherwise ``run`` evaluates the same
formulas with elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = {"mxfp8": 32, "nvfp4": 16}
KIND = {"mxfp8": 0, "nvfp4": 1}
LIMIT, ALPHA, OFFSET = 7.0, 1.702, 1.0   # clamped SwiGLU
GLU = ("glu", "glu_grad", "glu_gemv")


# ------------------------------------------------------------------ cases

def _case(name, op, recipe, experts, rows, n, k, act="swiglu", probs=True, groups=1, dtype="bf16"):
    """n: columns of the result; groups: how many groups the 2 n weight rows of an expert were quantized in."""
    c = {"name": name, "op": op, "recipe": recipe, "experts": experts, "rows": rows, "n": n, "k": k, "dtype": dtype}
    if op in GLU:
        c.update(act=act, probs=probs, groups=groups)
    return c


def listed():
    return [
        # a ragged batch with an output width that no tile divides, clamped
        _case("glu ragged mxfp8", "glu", "mxfp8", 16, 4999, 1000, 1024, "clamped_swiglu", True, 2),
        # four rows an expert: a short prefill, the experts' weights are what there is to read
        _case("glu few rows nvfp4", "glu", "nvfp4", 128, 512, 2048, 2048),
        # first projection of a training batch (32 experts, 65536 rows, width 2048)
        _case("glu train nvfp4", "glu", "nvfp4", 32, 65536, 2048, 2048),
        # first projection of the routed SwiGLU workload (262144 rows, width 4096): the largest
        _case("glu routed mxfp8", "glu", "mxfp8", 128, 262144, 4096, 2048),
        # gradient of the ragged batch
        _case("glu gradient ragged mxfp8", "glu_grad", "mxfp8", 16, 4999, 1000, 1024, "clamped_swiglu", True, 2),
        # gradient of the training batch
        _case("glu gradient train nvfp4", "glu_grad", "nvfp4", 32, 65536, 2048, 2048),
        # one token through one dense projection: launch and latency
        _case("gemv one token nvfp4", "gemv", "nvfp4", 1, 1, 4096, 4096),
        # four new tokens x top-8 through the second projection of 128 experts
        _case("gemv decode nvfp4", "gemv", "nvfp4", 128, 32, 2048, 4096),
        # odd sizes, FP32 rows and results
        _case("gemv odd fp32", "gemv", "nvfp4", 7, 20, 1111, 1088, dtype="fp32"),
        # a batch of sequences over eight experts, FP16
        _case("gemv batch mxfp8", "gemv", "mxfp8", 8, 64, 4096, 4096, dtype="fp16"),
        # one new token on its way through the first projection of its 8 experts
        _case("glu gemv one token nvfp4", "glu_gemv", "nvfp4", 128, 8, 4096, 2048),
        # eight new tokens x top-8, clamped
        _case("glu gemv decode mxfp8", "glu_gemv", "mxfp8", 128, 64, 2048, 2048, "clamped_swiglu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["glu", "glu_grad", "gemv", "glu_gemv"])
        recipe, groups = rng.choice(["mxfp8", "nvfp4"]), rng.choice([1, 2])
        k = 64 * _log(rng, 1, 64)
        if op in ("glu", "glu_grad"):
            e, m = _log(rng, 2, 128), _log(rng, 1, 262144)
            n = 128 * _log(rng, 1, 32) if groups == 1 else _log(rng, 16, 4096)
            big = 262144 * 4096 * 2048 if op == "glu" else 65536 * 2048 * 2048
            ok = m * n * k <= big // 2 and e * n * k <= (128 * 4096 * 2048 if op == "glu" else 64 * 2048 * 2048)
            dtype = "bf16"
        else:
            e = _log(rng, 1, 128)
            m = _log(rng, 1, 8 * e)
            n = 128 * _log(rng, 1, 32) if groups == 1 and op == "glu_gemv" else _log(rng, 16, 4096)
            ok = e * n * k <= 128 * 4096 * 2048
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if ok:
            c = _case("", op, recipe, e, m, n, k, rng.choice(["swiglu", "clamped_swiglu"]), rng.random() < 0.7, groups, dtype)
            del c["name"]
            return c


def _weights_of_experts(e):
    """Popularity of the experts: k^-1.1, the last e // 32 of them never chosen."""
    w = np.arange(1, e + 1, dtype=np.float64) ** -1.1
    w[e - e // 32:] = 0.0
    return w / w.sum()


def work(case):
    m, n, k, op = case["rows"], case["n"], case["k"], case["op"]
    per = (1.0 if case["recipe"] == "mxfp8" else 0.5) + 1.0 / BLOCK[case["recipe"]]
    rows_b = 2 * n if op in GLU else n
    active = float(np.sum(1 - (1 - _weights_of_experts(case["experts"])) ** m))
    size = SIZE[case["dtype"]]
    nbytes = active * rows_b * k * per + m * n * size + m * k * (per if op in ("glu", "glu_grad") else size)
    if op == "glu_grad":
        nbytes += m * 2 * n * size + 4 * m
    if case.get("probs"):
        nbytes += 4 * m
    return {"bytes": int(nbytes), "flops": 2 * m * rows_b * k}


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _split_rows(case, seed):
    rng = np.random.default_rng(int(seed) * 104729 + 7)
    w = rng.permutation(_weights_of_experts(case["experts"]))
    return [int(v) for v in rng.multinomial(case["rows"], w)]


def _e2m1(v):
    """E2M1 codes (uint8) of FP32 values in [-6, 6]: the nearest, a tie toward zero."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return (torch.bucketize(v.abs(), mid, out_int32=True) + 8 * (v < 0)).to(torch.uint8)


def _quantise(x, recipe, group, groups):
    """x [R, C] in blocks along C -> codes [R, C] (unpacked), scales [R, C / B], amax [groups]."""
    b = BLOCK[recipe]
    r, c = x.shape
    codes = torch.empty((r, c), dtype=torch.uint8, device=x.device)
    scales = torch.empty((r, c // b), dtype=torch.uint8, device=x.device)
    step = max(1, (1 << 26) // c)
    amax = torch.zeros(groups, device=x.device)
    if r:
        amax.scatter_reduce_(0, group, x.abs().amax(1), "amax")
    s_of = torch.where(amax > 0, 2688.0 / amax, torch.ones_like(amax))
    for r0 in range(0, r, step):
        v = x[r0:r0 + step].reshape(-1, c // b, b)
        m = v.abs().amax(2)
        if recipe == "nvfp4":
            s = s_of[group[r0:r0 + step]][:, None]
            s8 = (m / 6.0 * s).clamp_max(448.0).to(torch.float8_e4m3fn)
            f8 = s8.to(torch.float32)
            mult = torch.where(f8 > 0, s / f8, torch.zeros_like(f8))
            codes[r0:r0 + step] = _e2m1((v * mult[:, :, None]).clamp(-6.0, 6.0)).reshape(-1, c)
            scales[r0:r0 + step] = s8.view(torch.uint8)
        else:
            e = torch.ceil(torch.log2(m.clamp_min(1e-30) / 448.0)).clamp(-127, 127)
            q = (v * torch.exp2(-e)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            codes[r0:r0 + step] = q.view(torch.uint8).reshape(-1, c)
            scales[r0:r0 + step] = (e + 127).to(torch.uint8)
    return codes, scales, amax


def _row_copy(x, recipe, split):
    """The rowwise copy of x [M, C] grouped by split: packed codes, scales in tiles of 128 rows x 4, amax."""
    m, c = x.shape
    cb = c // BLOCK[recipe]
    group = torch.repeat_interleave(torch.arange(len(split), device=x.device), torch.tensor(split, device=x.device),
                                    output_size=m)
    codes, scales, amax = _quantise(x, recipe, group, len(split))
    tiles = [-(-s // 128) for s in split]
    c4 = -(-cb // 4)
    tiled = torch.zeros(max(1, sum(tiles)) * c4 * 512, dtype=torch.uint8, device=x.device)
    if m:
        row0 = torch.tensor(np.concatenate([[0], np.cumsum(split)[:-1]]), device=x.device)
        tile0 = torch.tensor(np.concatenate([[0], np.cumsum(tiles)[:-1]]), device=x.device)
        lr = torch.arange(m, device=x.device) - row0[group]
        col = torch.arange(cb, device=x.device)
        at = ((tile0[group] + lr // 128) * c4)[:, None] * 512 + (16 * (lr % 32) + 4 * (lr % 128 // 32))[:, None] + \
            (col // 4 * 512 + col % 4)[None, :]
        tiled[at] = scales
    if recipe == "nvfp4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return {"row_data": codes.reshape(-1), "row_scale": tiled, "amax_row": amax}


def prepare(case, seed):
    g = _generator(seed)
    e, m, n, k, recipe, op = (case[x] for x in ("experts", "rows", "n", "k", "recipe", "op"))
    split = _split_rows(case, seed)
    st = dict(case, split=torch.tensor(split, dtype=torch.int64, device="cuda"), split_host=split, p=None)
    groups, rows_b = (case["groups"], 2 * n) if op in GLU else (1, n)
    # pre-activations of a few units: the gate leaves its linear range, some linear values meet the clamp
    w = _normal(g, (e * rows_b, k)) * (2.5 / math.sqrt(k))
    st["b"] = _row_copy(w, recipe, [rows_b // groups] * (e * groups))
    del w
    x = _normal(g, (m, k))
    if op in ("glu", "glu_grad"):
        st["a"] = _row_copy(x, recipe, split)
    else:
        st["x"] = x.to(DTYPES[case["dtype"]])
    if case.get("probs"):
        st["p"] = torch.rand((m,), generator=g, device="cuda")
    if op == "glu_grad":
        st["dy"] = _normal(g, (m, n)).to(DTYPES[case["dtype"]])
    return st


# ------------------------------------------------------------- plain forms

def _values(data, recipe, shape):
    """FP32 values of packed codes laid out row by row."""
    if recipe == "mxfp8":
        return data.view(torch.float8_e4m3fn).reshape(shape).float()
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    return table[torch.stack((data & 15, data >> 4), -1).reshape(shape).int()]


def _scaled(q, recipe, values, tile, lr, unit):
    """values [..., k] of rows at local row lr of scale tile row `tile`, times block scales and unit (1 / S)."""
    cb = values.shape[-1] // BLOCK[recipe]
    c4 = -(-cb // 4)
    col = torch.arange(cb, device="cuda")
    at = (tile * c4 * 512 + 16 * (lr % 32) + 4 * (lr % 128 // 32))[..., None] + col // 4 * 512 + col % 4
    s = q["row_scale"][at]
    s = torch.exp2(s.float() - 127) if recipe == "mxfp8" else s.view(torch.float8_e4m3fn).float()
    v = (values.reshape(*values.shape[:-1], cb, -1) * s[..., None]).reshape(values.shape)
    return v if unit is None else v * unit[..., None]


def _unit(q, recipe):
    """1 / S of each group: what NVFP4's codes and block scales are relative to."""
    if recipe == "mxfp8":
        return None
    a = q["amax_row"]
    return torch.where(a > 0, a / 2688.0, torch.ones_like(a))


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda")


def _pieces(split):
    """Pieces of at most R rows of one expert: (expert, first row within it, R); R about the mean of the experts in use."""
    m = np.array(split)
    r = 1 << max(0, math.ceil(math.log2(max(1, m.sum() / max(1, (m > 0).sum())))))
    r = min(4096, r)
    pieces = -(-m // r)
    expert = np.repeat(np.arange(len(m)), pieces)
    first = (np.arange(len(expert)) - np.repeat(np.cumsum(pieces) - pieces, pieces)) * r
    return expert, first, r


def _rows_product(st, x, rows_b, groups):
    """x [m, k] FP32 against the weights [rows_b, k] of each row's expert: [m, rows_b] FP32."""
    m, k, recipe, b = st["rows"], st["k"], st["recipe"], st["b"]
    split = np.array(st["split_host"])
    row0 = np.cumsum(split) - split
    expert, first, r = _pieces(split)
    used, which = np.unique(expert, return_inverse=True)
    per = k if recipe == "mxfp8" else k // 2
    w = b["row_data"].reshape(-1, rows_b * per)[_dev(used)].reshape(-1)
    j = np.arange(rows_b)
    size = rows_b // groups
    group = used[:, None] * groups + j // size
    lr = j % size
    unit = _unit(b, recipe)
    w = _scaled(b, recipe, _values(w, recipe, (len(used), rows_b, k)), _dev(group * -(-size // 128) + lr // 128),
                _dev(np.broadcast_to(lr, group.shape)), None if unit is None else unit[_dev(group)])
    lrow = first[:, None] + np.arange(r)
    live = lrow < split[expert][:, None]
    at = _dev(np.where(live, row0[expert][:, None] + lrow, m))
    x = torch.cat((x, torch.zeros((1, k), device="cuda")))[at]
    y = torch.bmm(x, w[_dev(which)].transpose(1, 2)).reshape(-1, rows_b)
    return y[_dev(np.flatnonzero(live.reshape(-1)))]


def _pre_activations(st):
    if st["op"] == "glu_gemv":
        x = st["x"].float()
    else:
        m, k, recipe, a = st["rows"], st["k"], st["recipe"], st["a"]
        split = np.array(st["split_host"])
        tiles = -(-split // 128)
        expert = np.repeat(np.arange(len(split)), split)
        lr = np.arange(m) - (np.cumsum(split) - split)[expert]
        unit = _unit(a, recipe)
        x = _scaled(a, recipe, _values(a["row_data"], recipe, (m, k)), _dev((np.cumsum(tiles) - tiles)[expert] + lr // 128),
                    _dev(lr), None if unit is None else unit[_dev(expert)])
    h = _rows_product(st, x, 2 * st["n"], st["groups"])
    return h[:, :st["n"]], h[:, st["n"]:]


def _plain_glu(st):
    g, u = _pre_activations(st)
    if st["act"] == "swiglu":
        y = g * torch.sigmoid(g) * u
    else:
        g = g.clamp(max=LIMIT)
        y = g * torch.sigmoid(ALPHA * g) * (u.clamp(-LIMIT, LIMIT) + OFFSET)
    if st["p"] is not None:
        y = y * st["p"][:, None]
    return {"y": y.to(DTYPES[st["dtype"]])}


def _plain_glu_grad(st):
    g, u = _pre_activations(st)
    dy = st["dy"].float()
    t = dy if st["p"] is None else dy * st["p"][:, None]
    if st["act"] == "swiglu":
        s = torch.sigmoid(g)
        dprobs = (dy * (g * s * u)).sum(1)
        dg = t * u * (s + g * s * (1 - s))
        du = t * (g * s)
    else:
        a, b = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT) + OFFSET
        s = torch.sigmoid(ALPHA * a)
        dprobs = (dy * (a * s * b)).sum(1)
        dg = torch.where(g <= LIMIT, t * b * (s + ALPHA * a * s * (1 - s)), 0.0)
        du = torch.where(u.abs() <= LIMIT, t * (a * s), 0.0)
    return {"dx": torch.cat((dg, du), 1).to(DTYPES[st["dtype"]]), "dprobs": dprobs}


def _plain_gemv(st):
    return {"out": _rows_product(st, st["x"].float(), st["n"], 1).to(DTYPES[st["dtype"]])}


def _own(st):
    from nvfp4_quantization_grouped_gb300 import gsa
    op, n, k, kind = st["op"], st["n"], st["k"], KIND[st["recipe"]]
    if op == "gemv":
        return {"out": gsa.grouped_gemv(st["x"], st["b"], st["split"], n, kind)}
    act = {"act": st["act"], "probs": st["p"], "b_groups": st["groups"],
           "params": gsa.act_params(st["act"], limit=LIMIT, alpha=ALPHA, glu_linear_offset=OFFSET)}
    if op == "glu_gemv":
        return {"y": gsa.grouped_glu_gemv(st["x"], st["b"], st["split"], n, kind, **act)}
    if op == "glu":
        return {"y": gsa.grouped_glu(st["a"], st["b"], st["split"], st["rows"], n, k, kind, **act)}
    dx, dprobs = gsa.grouped_glu_bwd(st["dy"], st["a"], st["b"], st["split"], st["rows"], n, k, kind, **act)
    return {"dx": dx, "dprobs": dprobs}


def run(state):
    if own:
        return _own(state)
    return {"glu": _plain_glu, "glu_grad": _plain_glu_grad, "gemv": _plain_gemv, "glu_gemv": _plain_glu}[state["op"]](state)


# ------------------------------------------- the definitions in 64 bits

def _fp8_table():
    """Value of each E4M3 byte, from its fields."""
    v = []
    for c in range(256):
        s, e, f = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        v.append(math.nan if c & 127 == 127 else s * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)))
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _fp4_tables():
    """Value of the low and of the high nibble of each byte."""
    one = [(-1.0 if c & 8 else 1.0) * ((c & 1) / 2 if c & 6 == 0 else (1 + (c & 1) / 2) * 2.0 ** ((c >> 1 & 3) - 1))
           for c in range(16)]
    return [torch.tensor([one[c >> sh & 15] for c in range(256)], dtype=torch.float64, device="cuda") for sh in (0, 4)]


def _decode(data, scale, amax, recipe, rows, cols):
    """One quantized matrix [rows, cols]: codes row by row and its own 128 x 4 scale tiles, in FP64."""
    b = BLOCK[recipe]
    byte = data.reshape(rows, -1).int()
    if recipe == "mxfp8":
        v = _fp8_table()[byte]
    else:
        lo, hi = _fp4_tables()
        v = torch.empty((rows, cols), dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = lo[byte], hi[byte]
    t, c = -(-rows // 128), cols // b
    s = scale.reshape(t, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(t * 128, -1)[:rows, :c].int()
    s = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s - 127) if recipe == "mxfp8" else _fp8_table()[s]
    v = v * s.repeat_interleave(b, dim=1)
    if recipe == "nvfp4":
        v *= float(amax) / 2688.0 if float(amax) > 0 else 1.0
    return v


def exact(case, seed):
    if 2 * work(case)["flops"] > 3e13:   # minutes in 64 bits
        return None
    st = prepare(case, seed)
    n, k, recipe, op, m = st["n"], st["k"], st["recipe"], st["op"], st["rows"]
    groups, rows_b = (st["groups"], 2 * n) if op in GLU else (1, n)
    size, c4, half = rows_b // groups, -(-(k // BLOCK[recipe]) // 4) * 512, 1 if recipe == "mxfp8" else 2
    wd = st["b"]["row_data"].reshape(-1, size * k // half)
    ws = st["b"]["row_scale"].reshape(-1, -(-size // 128) * c4)
    h = torch.empty((m, rows_b), dtype=torch.float64, device="cuda")
    r = tile = 0
    for e, s in enumerate(st["split_host"]):
        t = -(-s // 128)
        if s:
            if "a" in st:
                x = _decode(st["a"]["row_data"][r * k // half:(r + s) * k // half], st["a"]["row_scale"][tile * c4:(tile + t) * c4],
                            st["a"]["amax_row"][e], recipe, s, k)
            else:
                x = st["x"][r:r + s].double()
            for j in range(e * groups, (e + 1) * groups):
                c = (j - e * groups) * size
                h[r:r + s, c:c + size] = x @ _decode(wd[j], ws[j], st["b"]["amax_row"][j], recipe, size, k).t()
        r, tile = r + s, tile + t
    if op == "gemv":
        return {"out": h}
    limit, alpha, offset = (math.inf, 1.0, 0.0) if st["act"] == "swiglu" else (LIMIT, ALPHA, OFFSET)
    gate, lin = h[:, :n], h[:, n:]
    a, b = torch.minimum(gate, torch.full_like(gate, limit)), lin.clamp(-limit, limit) + offset
    s = 1 / (1 + torch.exp(-alpha * a))
    v = a * s * b
    p = torch.ones(m, dtype=torch.float64, device="cuda") if st["p"] is None else st["p"].double()
    if op != "glu_grad":
        return {"y": v * p[:, None]}
    dy = st["dy"].double()
    dg = dy * p[:, None] * b * s * (1 + alpha * a * (1 - s)) * (gate <= limit)
    du = dy * p[:, None] * a * s * (lin.abs() <= limit)
    return {"dx": torch.cat((dg, du), 1), "dprobs": (dy * v).sum(1)}
