"""A call that CUDA refuses says so, and the next one does not find its error.  In a process of its own, since the
refused call is a status query of a stream under capture, which ends the capture."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
sys.path.insert(0, ".")
import torch
import attention_forward_02_gb300 as fa
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
dev = dict(device="cuda", dtype=torch.float16)
q, k = torch.randn(3, 4, 64, **dev), torch.randn(3, 2, 64, **dev)
rope = fa.FARope.new(64)
cache, pool = fa.FACache4.empty(4, 2, 16, 64), fa.FAPagePool.full(4)
table, lens, new, keep = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), i32([0]), i32([3]), i32([1])
plan = fa.fa_cache_plan(pool, table, lens, new, 16, 3)
cache8 = fa.FACache.empty(4, 2, 16, 64)
x = torch.randn(1, 2, 40, 64, **dev)

def calls():
    yield lambda: fa.fa_rope(q, k, rope, plan.positions, q_out=q, k_out=k)
    yield lambda: fa.fa_cache_plan(pool, table, lens, new, 16, 3, plan=plan)
    yield lambda: fa.fa_cache4_write(cache, k, k, plan.slots)
    yield lambda: fa.fa_cache4_read(cache, table, plan.ends, 3)
    yield lambda: fa.fa_decode_cache4(q.unsqueeze(2)[:1], cache, table, plan.ends)
    yield lambda: fa.fa_cache_trim(pool, table, plan.ends, keep, 16)
    yield lambda: fa.fa_cache_write(cache8, k, k, table, lens)
    yield lambda: fa.fa_decode_cache(q.unsqueeze(2)[:1], cache8, table, plan.ends)
    yield lambda: fa.fa_fwd(x, x, x)

for call in calls():
    call()
torch.cuda.synchronize()
for call in calls():
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        assert fa.fa_last_device_status(stream.cuda_stream) == 4
        try:
            graph.capture_end()
            raise SystemExit("the capture went on")
        except RuntimeError:
            pass
    call()
    torch.cuda.synchronize()
    print("good")
"""


def test_an_error_is_reported_once():
    done = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stdout + done.stderr
    assert done.stdout.split() == ["good"] * 9
