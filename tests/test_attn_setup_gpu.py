"""When the attention kernels are set up: not by a GEMV call, which does without them, and on the first attention call
also where that is being captured. Each case in a process of its own, since the library is set up once."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HEAD = """
import sys, time
import torch
from memory_bound_decode_gb300 import binding, inputs
from tests import attn_util as au
binding.lib()
W, x = inputs.weight(512, 512, seed=1, device="cuda"), inputs.activations(1, 512, seed=2, device="cuda")
y = torch.zeros((1, 512), device="cuda")
torch.cuda.synchronize()
def gemv():
    t = time.perf_counter()
    binding.gemv_bf16(W, x, y, 512, 512, 1, W.shape[1])
    return time.perf_counter() - t
lens = [700, 3, 0]
def attention(kind="bf16", dim=64):
    return au.Attn(lens, au.Cache(lens, 16, 2, dim, kind, seed=3), 8)
def status_calls():
    torch.cuda.synchronize()
    best = 1.0
    for _ in range(50):
        t = time.perf_counter()
        assert binding.gemv_device_status() == 0
        best = min(best, time.perf_counter() - t)
    return best
"""


def run(body):
    r = subprocess.run([sys.executable, "-c", HEAD + body], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.parametrize("mode", ["global", "thread_local"])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_first_attention_call_captured(kind, mode):
    """After nothing but a GEMV call."""
    run(f"""
gemv()
a = attention("{kind}")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, capture_error_mode="{mode}"):
    a.run()
for _ in range(2):
    a.guard.fill_(-777.0)
    g.replay()
    torch.cuda.synchronize()
    a.check()
assert binding.gemv_device_status() == 0
""")


def test_status_bits_without_and_with_attention():
    """The bits of the attention kernels are read once there has been an attention call, and a bad page is seen."""
    run("""
gemv()
alone = status_calls()
a = attention()
a.run()
torch.cuda.synchronize()
a.check()
both = status_calls()
assert alone < 0.8 * both, (alone, both)     # five words to copy, then eleven
a.cache.table.fill_(-1)
a.run()
torch.cuda.synchronize()
assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
assert binding.gemv_device_status() == 0
""")
