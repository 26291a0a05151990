"""No call touches memory outside its operands.

Each buffer of a call in turn lies in host memory that the GPU reads and writes through the host's page tables, once at
the end and once at the start of the only populated pages of a mapping: what the GPU touches beyond becomes resident."""
import ctypes
import mmap

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, NV, Matrices, padded
from test_gpu_moe_route import make_idx, plan

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

PAGE = mmap.PAGESIZE


@pytest.fixture(scope="module", autouse=True)
def pageable():
    torch.zeros(1, device="cuda")
    cuda, value = ctypes.CDLL("libcuda.so.1"), ctypes.c_int()
    for attribute in (88, 100):   # pageable memory access, by the host's page tables
        if cuda.cuDeviceGetAttribute(ctypes.byref(value), attribute, torch.cuda.current_device()) or not value.value:
            pytest.skip("the GPU does not use pageable host memory")


class Host:
    """The bytes of an array in a mapping, at the start of its populated pages or up to 16 bytes before their end."""

    def __init__(self, array, at_end):
        n = array.nbytes
        pages = -(-max(n, 1) // PAGE)
        margin = 64
        self.region = mmap.mmap(-1, (pages + 2 * margin) * PAGE, flags=mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS)
        self.region.madvise(mmap.MADV_NOHUGEPAGE)
        self.first = margin * PAGE + ((pages * PAGE - n) // 16 * 16 if at_end else 0)
        self.bytes = np.frombuffer(self.region, np.uint8)
        for p in range(pages):
            self.bytes[(margin + p) * PAGE] = 0
        self.bytes[self.first:self.first + n] = np.ascontiguousarray(array).reshape(-1).view(np.uint8)
        self.like, self.ptr, self.own = array, self.bytes.ctypes.data + self.first, slice(margin, margin + pages)

    def touched(self):
        flags = (ctypes.c_ubyte * (len(self.region) // PAGE))()
        assert ctypes.CDLL(None).mincore(ctypes.c_void_p(self.bytes.ctypes.data), ctypes.c_size_t(len(self.region)), flags) == 0
        resident = np.frombuffer(flags, np.uint8) & 1
        resident[self.own] = 0
        return np.flatnonzero(resident) - self.own.start

    def get(self):
        return self.bytes[self.first:self.first + self.like.nbytes].view(self.like.dtype).reshape(self.like.shape)


def run(call, inputs, outputs, check):
    """call(pointers by name); each buffer in host memory in turn, the others on the device."""
    for name in (*inputs, *outputs):
        for at_end in (True, False):
            host, dev = None, {}
            for k, v in (*inputs.items(), *outputs.items()):
                if k == name:
                    host = Host(v, at_end)
                else:
                    dev[k] = torch.from_numpy(v.reshape(-1).view(np.uint8)).cuda() if v.nbytes else torch.zeros(16, dtype=torch.uint8, device="cuda")
            assert call({k: host.ptr if k == name else dev[k].data_ptr() for k in (*inputs, *outputs)}) == 0
            torch.cuda.synchronize()
            assert host.touched().size == 0, (name, at_end, host.touched())
            check({k: host.get() if k == name else dev[k].cpu().numpy().view(v.dtype).reshape(v.shape) for k, v in outputs.items()})


def bits(rng, shape, dtype):
    v = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    return v.view(torch.int16 if v.element_size() == 2 else torch.int32).numpy()


TYPES = [(torch.bfloat16, gsa.BF16, np.int16), (torch.float16, gsa.FP16, np.int16), (torch.float32, gsa.FP32, np.int32)]
# widths of every access size, and rows of which several share a 16-byte word
SHAPES = [(37, 3, 1), (64, 2, 3), (130, 4, 2047), (96, 3, 1110), (33, 2, 1108), (40, 8, 512), (7, 5, 8200)]


@pytest.mark.parametrize("dtype,code,word", TYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,topk,hidden", SHAPES)
def test_row_moves(dtype, code, word, tokens, topk, hidden):
    rng = np.random.default_rng(hidden)
    row, _ = plan(make_idx(rng, tokens, topk, 6, 0.1), 6)
    n, live, at, L = tokens * topk, row >= 0, np.maximum(row, ~row), gsa.load()
    x, rows = bits(rng, (tokens, hidden), dtype), bits(rng, (n, hidden), dtype)
    probs, ps = rng.standard_normal((tokens, topk)).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    shape = (tokens, topk, hidden, code)

    def permuted(o):
        ref = np.zeros((n, hidden), word)
        ref[at[live]] = x[np.nonzero(live)[0]]
        assert np.array_equal(o["xs"], ref)

    run(lambda p: L.gsa_moe_permute(p["x"], p["probs"], p["row"], *shape, p["xs"], p["ps"], None),
        {"x": x, "probs": probs, "row": row}, {"xs": np.zeros((n, hidden), word), "ps": np.zeros(n, np.float32)}, permuted)
    first = {}

    def same(o):   # the results do not depend on where the buffers lie
        for k, v in o.items():
            assert np.array_equal(first.setdefault(k, v.copy()), v)

    run(lambda p: L.gsa_moe_permute_bwd(p["dxs"], p["dps"], p["row"], *shape, p["dx"], p["dprobs"], None),
        {"dxs": rows, "dps": ps, "row": row}, {"dx": np.zeros((tokens, hidden), word), "dprobs": np.zeros((tokens, topk), np.float32)}, same)
    first.clear()
    run(lambda p: L.gsa_moe_unpermute(p["ys"], p["w"], p["row"], *shape, p["out"], None),
        {"ys": rows, "w": probs, "row": row}, {"out": np.zeros((tokens, hidden), word)}, same)
    first.clear()
    run(lambda p: L.gsa_moe_unpermute_bwd(p["dout"], p["ys"], p["w"], p["row"], *shape, p["dys"], p["dw"], None),
        {"dout": x, "ys": rows, "w": probs, "row": row}, {"dys": np.zeros((n, hidden), word), "dw": np.zeros((tokens, topk), np.float32)}, same)


@pytest.mark.parametrize("tokens,topk", [(1, 1), (100, 3), (1365, 3), (4096, 1), (5001, 3), (100003, 1)])
def test_sort(tokens, topk):
    rng, L, experts = np.random.default_rng(tokens), gsa.load(), 37
    idx = make_idx(rng, tokens, topk, experts, 0.1)
    ref_row, ref_split = plan(idx, experts)
    nbytes = L.gsa_moe_sort_workspace_size(tokens, topk, experts)
    buffers = {"ws": np.zeros(nbytes, np.uint8)} if nbytes else {}

    def check(o):
        assert np.array_equal(o["row"], ref_row) and np.array_equal(o["split"], ref_split)

    run(lambda p: L.gsa_moe_sort(p["idx"], 8, tokens, topk, experts, p["row"], p["split"], p.get("ws"), nbytes, None),
        {"idx": idx, **buffers}, {"row": np.zeros((tokens, topk), np.int32), "split": np.zeros(experts + 1, np.int64)}, check)


def operand(p, side, m, scale):
    return gsa.QIn(p[side], p["s" + side], p["amax"], m.data.size - 1, scale.size)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", [([1], 1, 64), ([33, 97, 64, 1, 32], 100, 192), ([300, 17, 0, 64], 320, 576), ([600, 3], 260, 4160)], ids=str)
def test_product(recipe, split, n, k):
    rng, L, e, m = np.random.default_rng(k), gsa.load(), len(split), sum(split)
    a, b = Matrices(rng, split, k, recipe), Matrices(rng, [n] * e, k, recipe)
    ref = np.concatenate([x @ w.T for x, w in zip(a.values, b.values)])
    inputs = {"a": a.data[:-1], "b": b.data[:-1], "sa": a.scale, "sb": b.scale, "amax": a.amax, "split": np.array(split, np.int64)}

    def check(o):
        assert np.array_equal(o["out"].astype(np.float64), ref)

    run(lambda p: L.gsa_grouped_gemm(operand(p, "a", a, a.scale), operand(p, "b", b, b.scale), p["split"], e, m, n, k, recipe, p["out"], gsa.FP32, None),
        inputs, {"out": np.zeros((m, n), np.float32)}, check)


@pytest.mark.parametrize("recipe", [MX, NV])
@pytest.mark.parametrize("split,n,k", [([1], 2, 64), ([33, 97, 64, 1, 32], 100, 130), ([300, 17, 0, 64], 320, 512), ([2000, 3], 260, 134)], ids=str)
def test_weight_gradient(recipe, split, n, k):
    rng, L, e, m = np.random.default_rng(k), gsa.load(), len(split), sum(split)
    mp = padded(split, recipe)
    a, b = Matrices(rng, [n] * e, mp, recipe), Matrices(rng, [k] * e, mp, recipe)
    ref = np.stack([x @ w.T for x, w in zip(a.values, b.values)])
    nbytes = L.gsa_grouped_gemm_wgrad_workspace_size(e, m, n, k, recipe)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    inputs = {"a": a.data[:-1], "b": b.data[:-1], "sa": a.scale, "sb": b.scale, "amax": a.amax, "split": np.array(split, np.int64)}

    def check(o):
        assert np.array_equal(o["dw"].astype(np.float64), ref)

    run(lambda p: L.gsa_grouped_gemm_wgrad(operand(p, "a", a, a.scale), operand(p, "b", b, b.scale), p["split"], e, m, n, k, recipe, p["dw"],
                                           gsa.FP32, 0, ws.data_ptr(), nbytes, None),
        inputs, {"dw": np.zeros((e, n, k), np.float32)}, check)
