"""Workloads of the mixture-of-experts operators around the grouped activation.

Four operators, each in its training and serving forms:

* ``permute``    -- tokens sorted by expert: the sort plan of the routed expert
  indices and the gather of the token rows (and router probabilities) into
  expert order; its gradient adds the rows of a token's copies back together.
* ``unpermute``  -- the way back: the weighted sum of a token's expert rows; its
  gradient gives the rows' and the weights' gradients.
* ``product``    -- the grouped product of block-scaled (MXFP8 / NVFP4) rows with
  each expert's block-scaled weights, rows ragged over the experts.
* ``wgrad``      -- the weight gradient of that product: for each expert the
  product of two columnwise block-scaled copies over the expert's rows.

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


# ------------------------------------------------------------------ cases

def _route(name, op, way, tokens, topk, experts, hidden, dtype, drop=False):
    return {"name": name, "op": op, "way": way, "tokens": tokens, "topk": topk, "experts": experts, "hidden": hidden,
            "dtype": dtype, "drop": drop}


def _mm(name, op, recipe, experts, rows, n, k, out):
    return {"name": name, "op": op, "recipe": recipe, "experts": experts, "rows": rows, "n": n, "k": k, "out": out}


def listed():
    return [
        # a decode batch of 16 sequences on its way into 128 experts: launch latency is everything
        _route("permute decode", "permute", "fwd", 16, 8, 128, 4096, "bf16"),
        # the routed batch of the SwiGLU workload (32768 tokens x top-8, 128 experts): bandwidth
        _route("permute prefill", "permute", "fwd", 32768, 8, 128, 2048, "bf16"),
        # gradient with capacity drops, FP32 rows of an odd width that no vector access fits
        _route("permute gradient odd", "permute", "bwd", 5003, 3, 7, 1111, "fp32", True),
        # one new token coming back from its 8 experts
        _route("unpermute one token", "unpermute", "fwd", 1, 8, 128, 4096, "bf16"),
        # the way back of the routed batch
        _route("unpermute prefill", "unpermute", "fwd", 32768, 8, 128, 2048, "bf16"),
        # its training step on a quarter of the batch, with capacity drops
        _route("unpermute gradient", "unpermute", "bwd", 8192, 8, 128, 2048, "bf16", True),
        # four new tokens x top-8 through the second projection: a few rows, the active experts' weights are read
        _mm("product decode nvfp4", "product", "nvfp4", 128, 32, 2048, 4096, "bf16"),
        # second projection of the NVFP4 workload (32 experts, 65536 rows, width 2048)
        _mm("product train nvfp4", "product", "nvfp4", 32, 65536, 2048, 2048, "bf16"),
        # second projection of the routed SwiGLU workload (262144 rows, width 4096): the largest product
        _mm("product routed mxfp8", "product", "mxfp8", 128, 262144, 2048, 4096, "bf16"),
        # a ragged batch with an output width that no tile divides, FP32 results
        _mm("product ragged mxfp8", "product", "mxfp8", 16, 4999, 1000, 1024, "fp32"),
        # weight gradient of the NVFP4 workload's second projection, FP32 for the optimiser
        _mm("wgrad train nvfp4", "wgrad", "nvfp4", 32, 65536, 2048, 2048, "fp32"),
        # weight gradient of the 8-expert recompute workload (8192 rows, width 1024)
        _mm("wgrad small mxfp8", "wgrad", "mxfp8", 8, 8192, 1024, 1024, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["permute", "unpermute", "product", "wgrad"])
        if op in ("permute", "unpermute"):
            t, e = _log(rng, 1, 32768), _log(rng, 2, 256)
            k = rng.randint(1, min(8, e))
            h = _log(rng, 64, 4096)
            if rng.random() < 0.7:
                h = max(64, h // 8 * 8)
            c = _route("", op, rng.choice(["fwd", "bwd"]), t, k, e, h, rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                       rng.random() < 0.4)
            ok = t * k * h * SIZE[c["dtype"]] <= 32768 * 8 * 2048 * 2
        else:
            e, m = _log(rng, 2, 128), _log(rng, 1, 262144)
            n, k = 64 * _log(rng, 1, 64), 64 * _log(rng, 1, 64)
            if op == "product" and rng.random() < 0.4:
                n = max(1, n - rng.randint(1, 63))
            c = _mm("", op, rng.choice(["mxfp8", "nvfp4"]), e, m, n, k, rng.choice(["bf16", "bf16", "fp32"]))
            big = op == "product"
            ok = m * n * k <= (262144 * 4096 * 2048 if big else 65536 * 2048 * 2048) // 2 and \
                e * n * k <= (128 * 2048 * 4096 if big else 32 * 2048 * 2048)
        if ok:
            del c["name"]
            return c


def _weights_of_experts(e):
    """Popularity of the experts: k^-1.1, the last e // 32 of them never chosen."""
    w = np.arange(1, e + 1, dtype=np.float64) ** -1.1
    w[e - e // 32:] = 0.0
    return w / w.sum()


def _pad(m, b):
    return -(-m // b) * b


def work(case):
    if case["op"] in ("permute", "unpermute"):
        t, k, h, s = case["tokens"], case["topk"], case["hidden"], SIZE[case["dtype"]]
        small, large = t * h * s, t * k * h * s
        if case["op"] == "permute":
            # indices or plan, probabilities in and out, the token side once, the expert side once
            return {"bytes": small + large + t * k * (8 + 4 + 4 + 4), "flops": t * k * h if case["way"] == "bwd" else 0}
        if case["way"] == "fwd":
            return {"bytes": small + large + t * k * 8, "flops": 2 * t * k * h}
        return {"bytes": small + 2 * large + t * k * 12, "flops": 3 * t * k * h}
    m, n, k, b = case["rows"], case["n"], case["k"], BLOCK[case["recipe"]]
    o = SIZE[case["out"]]
    per = (1.0 if case["recipe"] == "mxfp8" else 0.5) + 1.0 / b
    if case["op"] == "product":
        active = float(np.sum(1 - (1 - _weights_of_experts(case["experts"])) ** m))
        return {"bytes": int(m * k * per + active * n * k * per + m * n * o), "flops": 2 * m * n * k}
    return {"bytes": int(m * (n + k) * per + case["experts"] * n * k * o), "flops": 2 * m * n * k}


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _expert_indices(g, case):
    """[tokens, topk] distinct experts a token (Gumbel top-k on the popularity); dropped slots hold -1."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    w = torch.from_numpy(_weights_of_experts(e)).to("cuda", torch.float32).clamp_min(1e-30)
    u = torch.rand((t, e), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
    idx = torch.topk(torch.log(w)[None, :] - torch.log(-torch.log(u)), k, dim=1).indices
    if case["drop"]:
        idx = torch.where(torch.rand((t, k), generator=g, device="cuda") < 0.05, -1, idx)
        idx[t // 2] = -1  # a token that no expert takes
    return idx


def _plan(idx, experts):
    """row_of_slot [T, topk] int32 and split [E + 1] int64: slots sorted by expert, in slot order within an
    expert; dropped slots come last, marked by the ones' complement of their row."""
    t, k = idx.shape
    key = torch.where((idx >= 0) & (idx < experts), idx, experts).reshape(-1)
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(t * k, device=idx.device)
    row = torch.where(key == experts, -1 - row, row).to(torch.int32).reshape(t, k)
    split = (key[:, None] == torch.arange(experts + 1, device=idx.device)[None, :]).sum(0)
    return row, split


def _split_rows(case, seed):
    rng = np.random.default_rng(int(seed) * 104729 + 7)
    w = rng.permutation(_weights_of_experts(case["experts"]))
    return [int(v) for v in rng.multinomial(case["rows"], w)]


def _e2m1(v):
    """E2M1 codes (uint8) of FP32 values in [-6, 6]: the nearest, a tie toward zero."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return (torch.bucketize(v.abs(), mid, out_int32=True) + 8 * (v < 0)).to(torch.uint8)


def _quantise(x, recipe, group, groups):
    """x [R, C] in blocks along C -> codes (MXFP8 [R, C] or NVFP4 [R, C] unpacked), scales [R, C / B], amax [groups]."""
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


def _col_copy(x, recipe, split):
    """The columnwise copy: for each expert the rowwise copy of its zero-padded transpose [C, Mp]."""
    m, c = x.shape
    b = BLOCK[recipe]
    data, scale, amax = [], [], []
    r0 = 0
    for s in split:
        mp = _pad(s, b)
        v = torch.zeros((mp, c), device=x.device)
        v[:s] = x[r0:r0 + s]
        r0 += s
        if s == 0:
            amax.append(torch.zeros(1, device=x.device))
            continue
        q = _row_copy(v.t().contiguous(), recipe, [c])
        data.append(q["row_data"])
        scale.append(q["row_scale"])
        amax.append(q["amax_row"])
    none = torch.zeros(1, dtype=torch.uint8, device=x.device)
    return {"col_data": torch.cat(data) if data else none, "col_scale": torch.cat(scale) if scale else none,
            "amax_col": torch.cat(amax)}


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    if case["op"] in ("permute", "unpermute"):
        t, k, e, h, dt = case["tokens"], case["topk"], case["experts"], case["hidden"], DTYPES[case["dtype"]]
        idx = _expert_indices(g, case)
        probs = torch.softmax(_normal(g, (t, k)), dim=1)
        if case["op"] == "permute" and case["way"] == "fwd":
            return {**st, "idx": idx, "x": _normal(g, (t, h), dt), "probs": probs}
        row, _ = _plan(idx, e)
        st["row_of_slot"] = row
        if case["op"] == "permute":
            return {**st, "dxs": _normal(g, (t * k, h), dt), "dps": _normal(g, (t * k,))}
        st.update(ys=_normal(g, (t * k, h), dt), weights=probs)
        if case["way"] == "bwd":
            st["dout"] = _normal(g, (t, h), dt)
        return st
    e, m, n, k, recipe = case["experts"], case["rows"], case["n"], case["k"], case["recipe"]
    split = _split_rows(case, seed)
    st.update(split=torch.tensor(split, dtype=torch.int64, device="cuda"), split_host=split)
    y = torch.relu(_normal(g, (m, k))).square_() * torch.rand((m, 1), generator=g, device="cuda")
    if case["op"] == "product":
        w = _normal(g, (e * n, k)) / math.sqrt(k)
        st.update(a=_row_copy(y, recipe, split), b=_row_copy(w, recipe, [n] * e))
    else:
        d = _normal(g, (m, n)) / 64
        st.update(a=_col_copy(d, recipe, split), b=_col_copy(y, recipe, split))
    return st


# ------------------------------------------------------------- plain forms

def _plain_permute(st):
    t, k, h = st["tokens"], st["topk"], st["hidden"]
    row, split = _plan(st["idx"], st["experts"])
    at = torch.where(row < 0, -1 - row, row).reshape(-1).long()
    live = (row >= 0).reshape(-1, 1)
    src = st["x"][:, None, :].expand(t, k, h).reshape(t * k, h)
    xs = torch.empty_like(src)
    xs[at] = torch.where(live, src, torch.zeros_like(src))
    ps = torch.empty(t * k, device=src.device)
    ps[at] = torch.where(live[:, 0], st["probs"].reshape(-1), 0.0)
    return {"row_of_slot": row, "split": split, "xs": xs, "ps": ps}


def _gather(rows, row):
    """rows[row] as [T, topk, H] in FP32, zeros for dropped slots."""
    live = row >= 0
    v = rows[torch.where(live, row, 0).long()].float()
    return torch.where(live[:, :, None], v, 0.0), live


def _plain_permute_grad(st):
    v, live = _gather(st["dxs"], st["row_of_slot"])
    dp, _ = _gather(st["dps"][:, None], st["row_of_slot"])
    return {"dx": v.sum(1).to(st["dxs"].dtype), "dprobs": dp[:, :, 0]}


def _plain_unpermute(st):
    v, _ = _gather(st["ys"], st["row_of_slot"])
    return {"out": (v * st["weights"][:, :, None]).sum(1).to(st["ys"].dtype)}


def _plain_unpermute_grad(st):
    row = st["row_of_slot"]
    v, live = _gather(st["ys"], row)
    d = st["dout"].float()
    dw = (v * d[:, None, :]).sum(2)
    g = torch.where(live[:, :, None], st["weights"][:, :, None] * d[:, None, :], 0.0).to(st["ys"].dtype)
    dys = torch.empty_like(st["ys"])
    dys[torch.where(live, row, -1 - row).reshape(-1).long()] = g.reshape(-1, g.shape[2])
    return {"dys": dys, "dweights": dw}


def _values(data, recipe, shape):
    """FP32 values of packed codes laid out row by row."""
    if recipe == "mxfp8":
        return data.view(torch.float8_e4m3fn).reshape(shape).float()
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    return table[torch.stack((data & 15, data >> 4), -1).reshape(shape).int()]


def _scale_values(scale, recipe):
    if recipe == "mxfp8":
        return torch.exp2(scale.float() - 127)
    return scale.view(torch.float8_e4m3fn).float()


def _unit(q, side, recipe):
    """1 / S of each expert: what NVFP4's codes and block scales are relative to."""
    if recipe == "mxfp8":
        return None
    a = q["amax_" + side]
    return torch.where(a > 0, a / 2688.0, torch.ones_like(a))


def _tiles(split, block=1):
    """Pieces of at most R rows of one expert: (expert, first row within it, R); R about the mean of the experts in use."""
    m = [_pad(s, block) for s in split]
    used = max(1, sum(s > 0 for s in m))
    r = 1 << max(0, math.ceil(math.log2(max(1, sum(m) / used))))
    r = min(4096, max(r, block))
    pieces = np.array([-(-s // r) for s in m])
    expert = np.repeat(np.arange(len(m)), pieces)
    first = (np.arange(len(expert)) - np.repeat(np.cumsum(pieces) - pieces, pieces)) * r
    return expert, first, r


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda")


def _plain_product(st):
    m, n, k, recipe, split = st["rows"], st["n"], st["k"], st["recipe"], st["split_host"]
    cb, c4 = k // BLOCK[recipe], -(-(k // BLOCK[recipe]) // 4)
    a, b = st["a"], st["b"]
    col = torch.arange(cb, device="cuda")
    col = col // 4 * 512 + col % 4

    def scaled(q, values, tile, lr):  # values [..., k] of rows at local row lr of scale tile `tile`
        at = (tile * c4 * 512 + 16 * (lr % 32) + 4 * (lr % 128 // 32))[..., None] + col
        s = _scale_values(q["row_scale"], recipe)[at]
        return (values.reshape(*values.shape[:-1], cb, -1) * s[..., None]).reshape(values.shape)

    split_np = np.array(split)
    row0, tile0 = np.cumsum(split_np) - split_np, np.cumsum(-(-split_np // 128)) - -(-split_np // 128)
    group = np.repeat(np.arange(len(split)), split_np)
    lr = np.arange(m) - row0[group]
    x = scaled(a, _values(a["row_data"], recipe, (m, k)), _dev(tile0[group] + lr // 128), _dev(lr))
    expert, first, r = _tiles(split)
    used, which = np.unique(expert, return_inverse=True)
    per = a["row_data"].numel() // max(1, m)
    w = b["row_data"].reshape(-1, n * per)[_dev(used)].reshape(-1)
    j = np.arange(n)
    w = scaled(b, _values(w, recipe, (len(used), n, k)), _dev(used[:, None] * -(-n // 128) + j // 128),
               _dev(np.broadcast_to(j, (len(used), n))))
    ua, ub = _unit(a, "row", recipe), _unit(b, "row", recipe)
    if ua is not None:
        x = x * ua[_dev(group)][:, None]
        w = w * ub[_dev(used)][:, None, None]
    lrow = first[:, None] + np.arange(r)
    live = lrow < split_np[expert][:, None]
    at = _dev(np.where(live, row0[expert][:, None] + lrow, m))
    x = torch.cat((x, torch.zeros((1, k), device="cuda")))[at]
    y = torch.bmm(x, w[_dev(which)].transpose(1, 2)).reshape(-1, n)
    return {"out": y[_dev(np.flatnonzero(live.reshape(-1)))].to(DTYPES[st["out"]])}


def _plain_wgrad(st):
    n, k, recipe, split = st["n"], st["k"], st["recipe"], np.array(st["split_host"])
    b = BLOCK[recipe]
    expert, first, r = _tiles(st["split_host"], b)
    mp = -(-split // b) * b
    pad0, sc0 = np.cumsum(mp) - mp, np.cumsum(-(-split // (4 * b))) - -(-split // (4 * b))
    lrow = first[:, None] + np.arange(r)  # padded row within the expert
    live = _dev(lrow < mp[expert][:, None])[:, None, :]
    lrow = np.minimum(lrow, np.maximum(mp[expert][:, None] - 1, 0))
    packed = 1 if recipe == "mxfp8" else 2

    def values(q, c):  # [pieces, c, r]
        j = torch.arange(c, device="cuda")[None, :, None]
        at = _dev(pad0[expert])[:, None, None] * c + j * _dev(mp[expert])[:, None, None] + _dev(lrow)[:, None, :]
        byte = q["col_data"][at // packed]
        if packed == 1:
            v = _values(byte, recipe, byte.shape)
        else:
            v = _values(torch.where(at % 2 == 1, byte >> 4, byte & 15)[..., None], recipe, (*byte.shape, 2))[..., 0]
        sb = _dev(lrow // b)[:, None, :]
        wide = _dev(-(-split[expert] // (4 * b)))[:, None, None]
        s_at = (_dev(sc0[expert])[:, None, None] * -(-c // 128) + j // 128 * wide + sb // 4) * 512 + \
            16 * (j % 32) + 4 * (j % 128 // 32) + sb % 4
        v = v * _scale_values(q["col_scale"], recipe)[s_at]
        u = _unit(q, "col", recipe)
        if u is not None:
            v = v * u[_dev(expert)][:, None, None]
        return torch.where(live, v, 0.0)

    part = torch.bmm(values(st["a"], n), values(st["b"], k).transpose(1, 2))
    dw = torch.zeros((len(split), n, k), device="cuda").index_add_(0, _dev(expert), part)
    return {"dw": dw.to(DTYPES[st["out"]])}


def _own(st):
    from nvfp4_quantization_grouped_gb300 import gsa
    op = st["op"]
    if op == "permute":
        if st["way"] == "fwd":
            row, split = gsa.moe_sort(st["idx"], st["experts"])
            xs, ps = gsa.moe_permute(st["x"], row, st["probs"])
            return {"row_of_slot": row, "split": split, "xs": xs, "ps": ps}
        dx, dprobs = gsa.moe_permute_bwd(st["dxs"], st["row_of_slot"], st["dps"])
        return {"dx": dx, "dprobs": dprobs}
    if op == "unpermute":
        if st["way"] == "fwd":
            return {"out": gsa.moe_unpermute(st["ys"], st["row_of_slot"], st["weights"])}
        dys, dw = gsa.moe_unpermute_bwd(st["dout"], st["ys"], st["row_of_slot"], st["weights"])
        return {"dys": dys, "dweights": dw}
    n, k, kind, dt = st["n"], st["k"], KIND[st["recipe"]], DTYPES[st["out"]]
    if op == "product":
        return {"out": gsa.grouped_gemm(st["a"], st["b"], st["split"], st["rows"], n, k, kind, out_dtype=dt)}
    return {"dw": gsa.grouped_gemm_wgrad(st["a"], st["b"], st["split"], st["rows"], n, k, kind, out_dtype=dt)}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "permute":
        return _plain_permute(state) if state["way"] == "fwd" else _plain_permute_grad(state)
    if state["op"] == "unpermute":
        return _plain_unpermute(state) if state["way"] == "fwd" else _plain_unpermute_grad(state)
    return _plain_product(state) if state["op"] == "product" else _plain_wgrad(state)


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
    """One quantised matrix [rows, cols]: codes row by row and its own 128 x 4 scale tiles, in FP64."""
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


def _exact_matrix(st):
    n, k, recipe, split = st["n"], st["k"], st["recipe"], st["split_host"]
    b, op = BLOCK[recipe], st["op"]
    a, w = st["a"], st["b"]
    half = 1 if recipe == "mxfp8" else 2
    outs = []
    r = da = sa = dw = sw = 0
    for e, s in enumerate(split):
        if op == "product":
            nd, ns = s * k // half, -(-s // 128) * -(-(k // b) // 4) * 512
            md, ms = n * k // half, -(-n // 128) * -(-(k // b) // 4) * 512
            if s:
                x = _decode(a["row_data"][da:da + nd], a["row_scale"][sa:sa + ns], a["amax_row"][e], recipe, s, k)
                y = _decode(w["row_data"][dw:dw + md], w["row_scale"][sw:sw + ms], w["amax_row"][e], recipe, n, k)
                outs.append(x @ y.t())
        else:
            mp, wide = _pad(s, b), -(-s // (4 * b))
            nd, ns = n * mp // half, -(-n // 128) * wide * 512
            md, ms = k * mp // half, -(-k // 128) * wide * 512
            if s:
                x = _decode(a["col_data"][da:da + nd], a["col_scale"][sa:sa + ns], a["amax_col"][e], recipe, n, mp)
                y = _decode(w["col_data"][dw:dw + md], w["col_scale"][sw:sw + ms], w["amax_col"][e], recipe, k, mp)
                outs.append(x @ y.t())
            else:
                outs.append(torch.zeros((n, k), dtype=torch.float64, device="cuda"))
        da, sa, dw, sw, r = da + nd, sa + ns, dw + md, sw + ms, r + s
    return {"out": torch.cat(outs)} if op == "product" else {"dw": torch.stack(outs)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("product", "wgrad"):
        return _exact_matrix(st)
    t, k, h, e = case["tokens"], case["topk"], case["hidden"], case["experts"]
    if case["op"] == "permute" and case["way"] == "fwd":
        idx = st["idx"].cpu().numpy().reshape(-1)
        idx = np.where((idx < 0) | (idx >= e), e, idx)
        slots = np.argsort(idx, kind="stable")  # the slot of each row
        row = np.empty(t * k, np.int64)
        row[slots] = np.arange(t * k)
        row = np.where(idx == e, ~row, row).reshape(t, k)
        keep = torch.from_numpy((idx[slots] < e).astype(np.float64)).cuda()
        token = torch.from_numpy(slots // k).cuda()
        return {"row_of_slot": torch.from_numpy(row.astype(np.int32)),
                "split": torch.from_numpy(np.bincount(idx, minlength=e + 1)),
                "xs": st["x"].double()[token] * keep[:, None],
                "ps": st["probs"].double().reshape(-1)[torch.from_numpy(slots).cuda()] * keep}
    row = st["row_of_slot"].long()
    live = (row >= 0).double()
    at = torch.maximum(row, ~row)
    if case["op"] == "permute":
        dx = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        for j in range(k):
            dx += st["dxs"][at[:, j]].double() * live[:, j:j + 1]
        return {"dx": dx, "dprobs": st["dps"].double()[at] * live}
    w = st["weights"].double() * live
    if case["way"] == "fwd":
        out = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        for j in range(k):
            out += st["ys"][at[:, j]].double() * w[:, j:j + 1]
        return {"out": out}
    d = st["dout"].double()
    dys = torch.empty((t * k, h), dtype=torch.float64, device="cuda")
    dw = torch.empty((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        dys[at[:, j]] = d * w[:, j:j + 1]
        dw[:, j] = (st["ys"][at[:, j]].double() * d).sum(1) * live[:, j]
    return {"dys": dys, "dweights": dw}
