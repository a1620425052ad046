"""gemv_rope_append into blocks whose scales are near FP32's largest number."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import blocks_cache as bc
from tests.test_append_blocks_gpu import check, run_and_check
from tests.test_rope_gpu import Case

pytestmark = pytest.mark.gpu

TOP = 2.0 ** 127
LARGEST = float(torch.finfo(torch.float32).max)         # (old / 2^127 below is exact)


def begun(old, new):
    """Blocks that hold every code but NaN under the scale `old`, and rows of values up to 2^127 for `new` tokens behind
    15 and 20 others."""
    cache = bc.BlockCache([15 + new, 20 + new], 32, 16, 4, 64, "head", seed=3)
    slots = cache.slots_of(0, 15, new) + cache.slots_of(1, 20, new)
    c = Case(len(slots), 4, 4, 64, 64, seed=3)
    c.k = torch.randn(c.k.shape, generator=torch.Generator().manual_seed(5)).clamp(-2, 2).cuda() * 2.0 ** 125
    c.v = torch.randn(c.v.shape, generator=torch.Generator().manual_seed(6)).clamp(-4, 4).cuda() * 2.0 ** 125
    for pool, scale in zip(cache.pools, cache.scales):
        scale.fill_(old)
        codes = torch.arange(pool.numel(), device="cuda").to(torch.uint8)
        pool.copy_(torch.where(codes & 0x7F == 0x7F, codes - 1, codes))
    return cache, slots, c


@pytest.mark.parametrize("new", [1, 5])                              # single tokens, runs
@pytest.mark.parametrize("old", [2.0 ** 120, 2.0 ** 125, 1.1 * 2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126, 1.99 * 2.0 ** 126, TOP])
def test_scales_up_to_the_largest_power(old, new):
    cache, slots, c = begun(old, new)
    run_and_check(c, cache, slots)


@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("old", [1.0001 * TOP, 1.5 * TOP, LARGEST])
def test_scales_past_the_largest_power(old, new):
    """They become 2^127; codes that have no place there are 448. The same call again changes nothing."""
    cache, slots, c = begun(old, new)
    before = cache.host()
    for codes, scales in before:
        for r, held in enumerate((15, 20)):
            slot = cache.slots_of(r, held, 1)[0]
            page, place = slot // 32, slot % 32
            at = cache.codes_of(codes)[page, place - held % 16:place]
            at.copy_(bc.code_of(at.contiguous().view(torch.float8_e4m3fn).float() * (old / TOP)).view(torch.uint8))
            cache.scales_of(scales)[page, place // 16] = TOP
    args = c.args(v=c.v, v_stride=c.sk, slots=torch.tensor(slots, dtype=torch.int32).cuda())
    for _ in range(2):
        binding.gemv_rope_append(args, cache.record())
        torch.cuda.synchronize()
        check(c, cache, slots, before, cache.host())
