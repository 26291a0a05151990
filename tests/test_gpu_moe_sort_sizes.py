"""The sort plan at the sizes where its kernels change (one warp's slots, one block's, a chunk of several steps a thread, the
first size of two launches), and from indices that start on no more than their own size."""
import numpy as np
import pytest
import torch

from test_gpu_moe_route import dev, make_idx, plan

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def check(idx, experts):
    row, split = gsa.moe_sort(idx, experts)
    ref_row, ref_split = plan(idx.cpu().numpy(), experts)
    assert np.array_equal(row.cpu().numpy(), ref_row)
    assert np.array_equal(split.cpu().numpy(), ref_split)


@pytest.mark.parametrize("slots", [31, 33, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 1024, 1025, 2047, 2049, 2500, 3072,
                                   4095, 4096, 4097, 6144, 8193])
@pytest.mark.parametrize("experts", [1, 40, 256])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sizes(slots, experts, drop):
    rng = np.random.default_rng(slots * 3 + experts)
    for topk in (1, 3, 7, 8):
        check(dev(make_idx(rng, slots // topk, topk, experts, drop)), experts)


@pytest.mark.parametrize("how", ["one expert", "all dropped", "sorted", "reversed"])
@pytest.mark.parametrize("tokens,topk", [(1500, 2), (1013, 3), (4096, 1), (1025, 1)])
def test_skewed_in_one_block(how, tokens, topk):
    experts, at = 40, np.arange(tokens * topk).reshape(tokens, topk)
    idx = {"one expert": np.full((tokens, topk), 17), "all dropped": np.full((tokens, topk), -1),
           "sorted": at * experts // at.size, "reversed": experts - 1 - at * experts // at.size}[how]
    check(dev(idx.astype(np.int64)), experts)


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("tokens", [5, 700, 3001, 50000])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_indices_that_start_anywhere(dtype, tokens, first):
    """Rows of a larger tensor: as a view from row `first` on they start on a multiple of their element's size."""
    rng = np.random.default_rng(tokens)
    for topk in (1, 3):
        check(dev(make_idx(rng, tokens + first, topk, 9, 0.1, dtype))[first:], 9)
