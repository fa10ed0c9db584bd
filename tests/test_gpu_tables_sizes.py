"""Sizes at which building block tables changes its kernel or its launch.  Whole numbers:
every comparison is exact."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

# n requests of one token each through a slot map of `cap` entries, in a process whose first
# call this is: what an earlier call with more requests asked for must not be needed.
ONE_CALL = """
import sys
sys.path[:0] = [{root!r}]
import torch, pagedattention_decode_03_b200 as pa
n, cap = {n}, {cap}
i32 = lambda k, v=0: torch.full((k,), v, dtype=torch.int32, device="cuda")
p = pa.pa_pool_create(num_layers=1, num_kv_heads=1, block_size=16, num_blocks=n, max_seqs=n, max_blocks_per_seq=1)
free, cu, slots, head, tables = torch.randperm(n).to(torch.int32).cuda(), i32(n + 1), i32(cap, -9), i32(1), i32(n, -7).view(n, 1)
pa.pa_build_tables(p, i32(n), i32(n, 1), free, head, head, tables, cu, slots)
assert pa.pa_check_device_errors(p) == 0
assert torch.equal(cu.cpu(), torch.arange(n + 1, dtype=torch.int32)) and int(head) == n
assert torch.equal(tables[:, 0], free) and torch.equal(slots[:n], free * 16) and bool((slots[n:] == -1).all())
"""


@pytest.mark.parametrize("n", [4072, 4073, 4095, 4096, 8192])
@pytest.mark.parametrize("cap", [9001, 400001])
def test_the_first_call_of_a_process(n, cap):
    """Sums of many requests take more shared memory than a launch has unasked."""
    r = subprocess.run([sys.executable, "-c", ONE_CALL.format(root=os.path.dirname(HERE), n=n, cap=cap)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
