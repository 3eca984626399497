"""fa_last_device_status costs a few round trips to the device, however many units have a status word."""
import time

import pytest
import torch

import attention_forward_02_gb300 as fa

pytestmark = pytest.mark.gpu


def least(call, times=30):
    best = float("inf")
    for _ in range(15):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        for _ in range(times):
            call()
        best = min(best, time.perf_counter() - begin)
    return best


def test_cost():
    """Reading the words one by one took seven times as long as reading one number back."""
    stream, x = torch.cuda.current_stream().cuda_stream, torch.zeros(1, device="cuda")
    for _ in range(5):  # other processes use the host too
        if least(lambda: fa.fa_last_device_status(stream)) < 4 * least(lambda: x.item()):
            return
    pytest.fail("a status query takes as long as four numbers read back")


def test_every_unit_s_word_is_read_and_cleared():
    """Bad pages and slots in each unit that reports them, on another stream, two units at once."""
    i32 = lambda n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(1, 1, 64, dtype=torch.float16, device="cuda")
    c8, c4 = fa.FACache.empty(2, 1, 16, 64), fa.FACache4.empty(2, 1, 16, 64)
    pool, table = fa.FAPagePool.full(2), torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    calls = [lambda: fa.fa_cache_write(c8, x, x, table + 9, i32([0])), lambda: fa.fa_cache4_write(c4, x, x, i32([99])),
             lambda: fa.fa_cache_plan(pool, table, i32([-1]), i32([1]), 16, 1, counts=pool.counts.clone())]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        handle = stream.cuda_stream
        assert fa.fa_last_device_status(handle) == 0
        for i, call in enumerate(calls):
            call()
            calls[i - 1]()
            assert fa.fa_last_device_status(handle) == 6
            assert fa.fa_last_device_status(handle) == 0
        assert fa.fa_selftest_wait_timeout(500, handle) == 0
        assert fa.fa_last_device_status(handle) == 5
        assert fa.fa_last_device_status(handle) == 0
