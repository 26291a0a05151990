"""The status query of the grouped products beside another thread that asks too."""
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
    return a.dev(), b.dev(), n, k


def test_no_report_is_lost_to_a_concurrent_query():
    """Every bad split is seen by the query behind it on its stream, or by one that another thread made meanwhile."""
    a, b, n, k = problem()
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
