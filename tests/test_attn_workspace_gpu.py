"""gemv_attn_decode's workspace: what is refused as too small, on the host, before anything is launched."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_too_small_for_the_shape(kind):
    """The workspace of 32 heads on 8 KV heads of 128 does not do for 32 on one: refused, and nothing is written."""
    few = binding.attn_workspace(32, 8, 128)
    lens = [300, 40]
    cache = au.Cache(lens, 16, 1, 128, kind, seed=3)
    need = binding.attn_workspace(32, 1, 128).nbytes
    assert few.nbytes < need
    for ws in (few, torch.zeros(need - 16, dtype=torch.uint8, device="cuda")):
        a = au.Attn(lens, cache, 32, workspace=ws)
        with pytest.raises(binding.GemvError) as e:
            a.run()
        assert e.value.status == binding.GEMV_ERR_INVALID
        torch.cuda.synchronize()
        assert (a.guard.float() == float(torch.tensor(-777.0).bfloat16())).all() and (ws == 0).all()
    a = au.Attn(lens, cache, 32, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_larger_than_needed():
    """The larger layout's workspace serves the smaller one, in turn."""
    ws = binding.attn_workspace(32, 1, 128)
    for heads in (1, 8, 1, 2):
        lens = [700, 3, 5000]
        a = au.Attn(lens, au.Cache(lens, 16, heads, 128, seed=heads), 32, workspace=ws)
        a.run()
        torch.cuda.synchronize()
        a.check()
