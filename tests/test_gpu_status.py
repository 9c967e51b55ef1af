"""sta_device_status(): what it costs, and records of both kinds at once."""
import ctypes
import time

import pytest
import torch

import block_sparse_local_b200 as sta
from block_sparse_local_b200 import workloads
from tests import kv_cases

pytestmark = pytest.mark.gpu


def _median_us(call, repeats=41, count=100):
    times = []
    for _ in range(repeats):
        t = time.perf_counter()
        for _ in range(count):
            call()
        times.append((time.perf_counter() - t) / count * 1e6)
    return sorted(times)[repeats // 2]


def test_the_call_costs_one_small_copy():
    # both records come back in one copy: with two the call takes twice as long
    # (18.7 us, 9.9 with one), half as much again is the border
    L = sta.lib()
    rt = ctypes.CDLL("libcudart.so.12")
    rt.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    rt.cudaStreamSynchronize.argtypes = [ctypes.c_void_p]
    x, host = torch.zeros(2, dtype=torch.int32, device="cuda"), (ctypes.c_int * 2)()
    src, dst = x.data_ptr(), ctypes.addressof(host)

    def copy():
        rt.cudaStreamSynchronize(None)
        assert rt.cudaMemcpy(dst, src, 8, 2) == 0

    assert L.sta_device_status(None) == 0
    copy()
    best = min(_median_us(lambda: L.sta_device_status(None)) / _median_us(copy) for _ in range(3))
    assert best < 1.5, best


def test_an_index_out_of_range_and_a_wait_that_gave_up():
    L = sta.lib()
    w = workloads.small_sta_case(12, 16, 24, (6, 8, 8), [(2, 2, 2)], 50, True, d=128, seed=29)
    q, k, v = (x.cuda() for x in workloads.sta_inputs(w))
    assert L.sta_debug_inject(1, 50) == 0      # a load that is left out; the wait ends
    try:
        sta.forward_raster(q, k, v, w.windows, w.text_len, w.has_text, (w.T, w.H, w.W), w.tile)
        kc, vc, _, _ = sta.kv_cache_empty(2, 1, 16, 64)
        x = torch.ones((2, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
        sta.kv_cache_append(x, x, kc, vc, kv_cases.i32([[2], [1]]), kv_cases.i32([1, 1]))
        codes = [L.sta_device_status(None) for _ in range(3)]
    finally:
        assert L.sta_debug_inject(0, 2000) == 0
    assert codes == [6, 4, 0]                  # each reported once
    assert kc[1, 0, 0].eq(1).all() and not kc[0].any()
