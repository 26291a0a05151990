"""The status query of the grouped products beside other threads: one that captures a graph, and one that asks too."""
import threading
import time

import numpy as np
import pytest
import torch

from test_gpu_grouped_gemm import MX, Matrices, dev_split

from nvfp4_quantization_grouped_gb300 import gsa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def problem():
    rng = np.random.default_rng(21)
    split, n, k = [10, 20], 64, 128
    a, b = Matrices(rng, split, k, MX), Matrices(rng, [n] * 2, k, MX)
    ref = np.concatenate([x @ w.T for x, w in zip(a.values, b.values)])
    return a.dev(), b.dev(), split, n, k, ref


def test_query_beside_another_threads_capture():
    a, b, split, n, k, ref = problem()
    s, side, seen = dev_split(split), torch.cuda.Stream(), []
    gsa.grouped_gemm_status(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):   # the mode that forbids unsafe calls to every thread
        out = gsa.grouped_gemm(a, b, s, 30, n, k, MX, out_dtype=torch.float32)
        t = threading.Thread(target=lambda: seen.append(gsa.grouped_gemm_status(side)))
        t.start()
        t.join()
    assert seen == [0]
    graph.replay()
    assert np.array_equal(out.double().cpu().numpy(), ref)


def test_query_of_a_capturing_stream_leaves_the_capture_alone():
    a, b, split, n, k, ref = problem()
    s = dev_split(split)
    gsa.grouped_gemm_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gsa.grouped_gemm(a, b, s, 30, n, k, MX, out_dtype=torch.float32)
        assert gsa.grouped_gemm_status() == 5   # GSA_ERR_CUDA: cannot be asked here
    graph.replay()
    assert np.array_equal(out.double().cpu().numpy(), ref)
    assert gsa.grouped_gemm_status() == 0


def test_no_report_is_lost_to_a_concurrent_query():
    """Every bad split is seen by the query behind it on its stream, or by one that another thread made meanwhile."""
    a, b, split, n, k, _ = problem()
    bad, out = dev_split([10, 21]), torch.empty((30, n), device="cuda")
    side, lock, stop, other = torch.cuda.Stream(), threading.Lock(), threading.Event(), [0]
    gsa.grouped_gemm_status()

    def ask():
        while not stop.is_set():
            with lock:
                other[0] += gsa.grouped_gemm_status(side) == 1
            time.sleep(0)   # the lock goes round

    t = threading.Thread(target=ask)
    t.start()
    lost = twice = 0
    try:
        for _ in range(1000):
            before = other[0]
            gsa.grouped_gemm(a, b, bad, 30, n, k, MX, out=out)
            mine = gsa.grouped_gemm_status()
            with lock:   # the other query under way has been counted
                theirs = other[0] - before
            lost += mine == 0 and theirs == 0
            twice += mine == 1 and theirs > 0
    finally:
        stop.set()
        t.join()
    assert gsa.grouped_gemm_status() == 0
    assert (lost, twice) == (0, 0)
