"""The status words that ra_sync_status reads: of the kernels that a program has used."""
import subprocess
import sys

import pytest

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from torch.profiler import ProfilerActivity, profile
import int4_quantized_flashattention_b200 as ra

def copies():
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        assert ra.sync_status() == 0
        torch.cuda.synchronize()
    return sum(e.count for e in p.key_averages() if e.key.startswith("Memcpy"))

p = ra.Problem.make(1, 2, 64, (24, 20, 20), (1, 4, 4), rot=0)
x = torch.zeros(1, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
pos = torch.zeros(16, 3, device="cuda", dtype=torch.int32)
copies()
ra.rope_bf16(p, x, x, pos)
old = copies()
ra.qk_norm_rope(p, x, x, None, None)
one = copies()
c = ra.KV4Cache.empty(1, 16, 2, 64)
table = torch.zeros(1, 1, device="cuda", dtype=torch.int32)
ra.kv4_append(c, x, x, table)
two = copies()
lens = torch.full((1,), 16, device="cuda", dtype=torch.int32)
ra.attn_cross(x, x, x)
three = copies()
print("copies", old, one, two, three)
# what each of them reports still arrives
table.fill_(7)
ra.kv4_append(c, x, x, table)
assert ra.sync_status() == 1
ra.attn_cross(x, x, x, lens + 1)
assert ra.sync_status() == 1
pos.fill_(9)
ra.qk_norm_rope(p, x, x, ra.rope_table(p), pos)
assert ra.sync_status() == 1 and ra.sync_status() == 0
"""


def test_only_kernels_in_use_are_asked():
    gu.device()
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=300,
                       cwd=__graft_entry__.ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    old, one, two, three = (int(n) for n in r.stdout.split("copies")[1].split())
    # a read and a clearing write per status word: four words of the older kernels
    assert old == 8 and one == 10 and two == 12 and three == 14
