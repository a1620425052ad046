"""When the kernels of attention over a cache with a scale for each block are set up: not by calls over the other caches, which
do without them, and on the first such call also where that is being captured. Each case in a process of its own."""
import pytest

from tests.test_attn_setup_gpu import run

pytestmark = pytest.mark.gpu

BLOCKS = """
from tests import blocks_cache as bc
from tests.test_attn_blocks_gpu import Attn
def over_blocks():
    return Attn(lens, bc.BlockCache(lens, 16, 16, 2, 64, seed=3), 8)
def taken(a):
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    a.run()
    torch.cuda.synchronize()
    after = torch.cuda.mem_get_info()[0]
    a.check()
    return before - after
"""


def test_other_caches_do_without():
    """Device memory (the kernels': some 2 MB) is taken by the first call over each, and gemv_device_status copies words of
    the kernels in use alone: five, then eleven, then fourteen."""
    run(BLOCKS + """
gemv()
a, b = attention(), over_blocks()
assert taken(a) > 0
others = status_calls()
assert taken(b) > 0, "loaded with the others"
both = status_calls()
assert others < 0.93 * both, (others, both)
assert taken(a) == 0 and taken(b) == 0
""")


@pytest.mark.parametrize("mode", ["global", "thread_local"])
@pytest.mark.parametrize("first", ["gemv()", "attention().run()"])
def test_first_call_captured(first, mode):
    run(BLOCKS + f"""
{first}
a = over_blocks()
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


@pytest.mark.parametrize("first", ["gemv()", "attention().run()"])
def test_status_bits(first):
    run(BLOCKS + f"""
{first}
a = over_blocks()
a.cache.table.fill_(-1)
a.run()
torch.cuda.synchronize()
assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
assert binding.gemv_device_status() == 0
b = attention()
b.cache.table.fill_(-1)
b.run()
torch.cuda.synchronize()
assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
assert binding.gemv_device_status() == 0
""")
