"""A cache with a scale for each block of tokens and head whose scales go to the
ends of FP32: attention over them, against 64 bits."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import blocks_cache as bc
from tests.test_attn_blocks_gpu import Attn

pytestmark = pytest.mark.gpu

LARGEST = float(torch.finfo(torch.float32).max)


class Wide(Attn):
    """BF16 ends below 2^128: what rounds there is an infinity. Taken as the 2^128 that one more exponent would hold
    (every value from 2^128 - 2^119 to 2^128 + 2^120 rounds to it), it is off by the same half step as the rest."""

    def check(self):
        stored, wide = self.guard, self.guard.double()
        self.guard = torch.where(wide.isinf(), wide.sign() * 2.0 ** 128, wide)
        super().check()
        self.guard = stored


def rescaled(cache, lens, scale_of, seed):
    """v's codes of 1/4 to 1 in magnitude (none of them 0, and values within FP32's range) and the scale
    scale_of(r, b) for block b of request r; k's scales where scores are moderate."""
    g = torch.Generator().manual_seed(seed)
    for i in range(2):
        pool, scale = cache.pools[i].cpu(), cache.scales[i].cpu()
        codes, scales = cache.codes_of(pool), cache.scales_of(scale)
        for r, n in enumerate(lens):
            x = torch.rand(n, cache.heads, cache.dim, generator=g) * 0.75 + 0.25
            x = bc.code_of(x * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1))
            for b in range(-(-n // cache.block)):
                j = slice(b * cache.block, min(n, (b + 1) * cache.block))
                page, place = int(cache.host_table[r, j.start // cache.page]), j.start % cache.page
                at = codes[page, place:place + j.stop - j.start]
                s = torch.tensor(scale_of(r, b) if i else 2.0 ** -6)
                if i:
                    at.copy_(x[j].view(torch.uint8))
                scales[page, place // cache.block] = s
                cache.values[i][r][j] = at.contiguous().view(torch.float8_e4m3fn).double() * float(s)
        cache.pools[i].copy_(pool)
        cache.scales[i].copy_(scale)


SHAPES = [
    # page, block, q_heads, heads, dim, lens
    (16, 16, 8, 2, 64, [1000, 17, 1, 0]),
    (64, 64, 8, 2, 128, [20000]),              # rows cut between CTAs
    (7, 7, 6, 1, 128, [400, 8]),               # copies by every thread
    (24, 8, 32, 2, 256, [2500, 50]),
    (32, 1, 64, 2, 64, [700, 33]),
    (128, 64, 5, 5, 96, [129, 1, 600]),
]


def run(shape, scale_of):
    page, block, q_heads, heads, dim, lens = shape
    cache = bc.BlockCache(lens, page, block, heads, dim, seed=page)
    rescaled(cache, lens, scale_of, seed=dim)
    a = Wide(lens, cache, q_heads, seed=3)
    for _ in range(2):
        a.run()
        torch.cuda.synchronize()
        a.check()
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 126, 1.3 * 2.0 ** 126, 2.0 ** 127, 1.9 * 2.0 ** 127, LARGEST])
def test_scales_at_the_top(shape, scale):
    """One over such a scale is subnormal from 2^126 on: the sum of weights must not lose it."""
    run(shape, lambda r, b: scale)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("low,high", [(-30, 120), (-60, 120), (-60, 127), (-20, 127), (-60, 60)])
@pytest.mark.parametrize("every", [1 << 20, 9])
def test_one_block_far_above_the_others(shape, low, high, every):
    """The products of one block, here and there, are by 2^high / 2^low the largest, but the probabilities of the
    others stay in the sum that they are divided by. The first of them comes early in the row or late."""
    for at in (0, 7):
        run(shape, lambda r, b: 2.0 ** (high if b % every == at % every else low))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("up", [False, True])
def test_scales_that_climb_and_fall(shape, up):
    """The running maximum moves by up to 2^180, in steps; rows are cut between warps and CTAs along the way."""
    last = max(shape[5]) // shape[1]
    run(shape, lambda r, b: 2.0 ** round(-60 + 187 * ((b if up else last - b) / max(1, last))))
