"""gemv_attn_decode over a cache with a scale for each block of tokens and head,
against 64 bits."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au
from tests import blocks_cache as bc

pytestmark = pytest.mark.gpu

# On top of an FP8 cache's bounds: log2 of v's scale is off by 2^-22 of itself (below 2^-17 in the exponent of a weight
# for scales of 2^-40 to 2^40) and its sum with the score by a rounding of at most 2^-24 of either.
MORE = 2.0 ** -17


class Attn(au.Attn):
    def check(self, lens=None):
        lens = self.lens if lens is None else lens
        Hq, D = self.q_heads, self.cache.dim
        got, mark = self.guard.double().cpu(), float(torch.tensor(-777.0).bfloat16())
        lse = self.lse.double().cpu() if self.lse is not None else None
        assert (got[0] == mark).all() and (got[-1] == mark).all() and (got[1:-1, Hq * D:] == mark).all()
        for r, n in enumerate(lens):
            y = got[1 + r, :Hq * D].view(Hq, D)
            if n < 0:
                assert (y == mark).all()
                continue
            if n == 0:
                assert (y == 0).all() and (lse is None or (lse[r] == -math.inf).all())
                continue
            begin = max(0, n - self.window) if self.window else 0
            k, v = (self.cache.values[i][r][begin:n] for i in range(2))
            q = self.q[r, :Hq * D].cpu().view(Hq, D)
            out, z, mass, size = au.attend(q, k, v, self.scale, self.softcap)
            tol, tol_z = au.attn_bounds(out, z, mass, size, n - begin, D, "fp8")
            err = (y - out).abs()
            tol = tol + 2 * MORE * mass
            assert (err <= tol).all(), (r, n, float((err / tol).max()))
            if lse is not None:
                assert ((lse[r] - z).abs() <= tol_z + MORE).all(), (r, n, float((lse[r] - z).abs().max()))


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page,block,q_heads,heads,dim,lens,window,softcap", [
    (16, 16, 32, 8, 128, [1, 15, 16, 17, 1000, 0, -1], 0, 0.0),
    (64, 32, 32, 8, 128, [64, 63, 65, 4001], 0, 0.0),
    (64, 64, 16, 2, 64, [130, 3000, 5], 100, 0.0),
    (24, 8, 32, 2, 256, [9000, 23, 24, 25], 4096, 50.0),
    (24, 24, 10, 2, 80, [700, 48, 0], 0, 30.0),
    (1, 1, 8, 4, 96, [77, 300], 0, 0.0),
    (7, 7, 6, 1, 128, [200, 6, 7], 50, 0.0),
    (32, 1, 64, 2, 128, [500, 33], 0, 0.0),
    (128, 64, 40, 1, 128, [5000, 127], 0, 0.0),
    (128, 16, 5, 5, 256, [129, 1], 0, 0.0),
])
def test_attention(layout, page, block, q_heads, heads, dim, lens, window, softcap):
    cache = bc.BlockCache(lens, page, block, heads, dim, layout, seed=page + block, extra=16, powers=block != 16)
    a = Attn(lens, cache, q_heads, seed=dim, window=window, softcap=softcap, pad=4)
    for _ in range(2):                             # the workspace is fit for the next call
        a.run()
        torch.cuda.synchronize()
        a.check()
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("requests,length", [(1, 40000), (40, 700), (300, 90), (64, 2048)])
def test_work_split(requests, length):
    """One long row, rows cut between CTAs, more requests than threads."""
    lens = [length] * requests if requests != 300 else [(r * 13) % length for r in range(requests)]
    cache = bc.BlockCache(lens, 32, 32, 2, 64, "head", seed=requests)
    a = Attn(lens, cache, 8, seed=3)
    a.run()
    torch.cuda.synchronize()
    a.check()
    first = a.guard.clone()
    a.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), a.guard.view(torch.int16)), "the same bits"


@pytest.mark.parametrize("requests,heads", [(2, 8), (16, 8), (32, 1), (33, 2), (100, 6), (256, 4), (257, 2)])
@pytest.mark.parametrize("longest", [1, 64, 130, 1024, 1025])
def test_rows_taken_whole(requests, heads, longest):
    """Ragged rows on both sides of the lengths, and numbers of requests, up to which a CTA takes whole ones."""
    if requests * longest * heads > 700000:
        pytest.skip("the reference takes long")
    g = torch.Generator().manual_seed(requests + longest)
    lens = torch.randint(0, longest + 1, (requests,), generator=g).tolist()
    lens[requests // 2] = longest
    lens[0] = 0
    cache = bc.BlockCache(lens, 64, 16, heads, 64, "head", seed=longest)
    a = Attn(lens, cache, 2 * heads, seed=3)
    a.run()
    torch.cuda.synchronize()
    a.check()


@pytest.mark.parametrize("spread", [(-40, 40), (-25, -20), (20, 25), (-3, 3)])
def test_scales_far_apart(spread):
    """v's blocks differ by up to 2^80: weights are relative to the largest product, so the bound holds throughout."""
    lens = [500, 40, 17]
    cache = bc.BlockCache(lens, 16, 16, 4, 64, seed=7, spread=spread)
    for i in range(1):                             # k stays where scores are moderate
        s = cache.scales_of(cache.scales[i].cpu())
        for r, n in enumerate(lens):
            v = torch.zeros(n, 4, 64, dtype=torch.float64)
            for j in range(n):
                slot = cache.slots_of(r, j, 1)[0]
                s[slot // 16, slot % 16 // 16] = 2.0 ** -6
                code = cache.codes_of(cache.pools[i].cpu())[slot // 16, slot % 16].contiguous().view(torch.float8_e4m3fn)
                v[j] = code.double() * 2.0 ** -6
            cache.values[i][r] = v
        cache.scales[i].copy_(s.as_strided((cache.scales[i].numel(),), (1,)))
    a = Attn(lens, cache, 8, seed=3)
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_blocks_of_zeros_with_a_scale_of_zero():
    lens = [70]
    cache = bc.BlockCache(lens, 16, 16, 2, 64, "token", seed=8)
    for i in range(2):
        pool, scale = cache.pools[i].cpu(), cache.scales[i].cpu()
        for blk in (0, 3):
            page = int(cache.host_table[0, blk])
            cache.codes_of(pool)[page] = 0
            cache.scales_of(scale)[page] = 0.0
            cache.values[i][0][blk * 16:blk * 16 + 16] = 0.0
        cache.pools[i].copy_(pool)
        cache.scales[i].copy_(scale)
    a = Attn(lens, cache, 8, seed=3)
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_nothing_but_zeros_under_scales_of_zero():
    """Every scale of v 0, many tokens: the sum of weights stays in range, the log-sum-exp is k's."""
    lens = [9000]
    cache = bc.BlockCache(lens, 64, 64, 2, 64, "head", seed=8)
    cache.pools[1].zero_()
    cache.scales[1].zero_()
    cache.values[1][0].zero_()
    a = Attn(lens, cache, 8, seed=3)
    a.run()
    torch.cuda.synchronize()
    a.check()
    assert (a.out == 0).all()


def test_scales_that_are_no_numbers_reach_their_own_head_only():
    lens = [40, 40]
    cache = bc.BlockCache(lens, 16, 16, 2, 64, "token", seed=9)
    for i, bad in ((0, math.nan), (1, math.nan)):
        a = Attn(lens, cache, 4, seed=3)
        scale = cache.scales[i].cpu()
        page = int(cache.host_table[1, 1])
        keep = cache.scales_of(scale)[page, 0, 1].clone()
        cache.scales_of(scale)[page, 0, 1] = bad
        cache.scales[i].copy_(scale)
        a.run()
        torch.cuda.synchronize()
        out = a.out.float().cpu().view(2, 4, 64)
        assert out[0].isfinite().all() and out[1, :2].isfinite().all() and out[1, 2:].isnan().all()
        assert a.lse[1, 2:].isnan().all() and a.lse[1, :2].isfinite().all()
        cache.scales_of(scale)[page, 0, 1] = keep
        cache.scales[i].copy_(scale)


def test_page_outside_the_pool():
    """Its tokens count as masked, its scales are not read."""
    lens = [64, 10]
    cache = bc.BlockCache(lens, 16, 16, 2, 64, "token", seed=9)
    table = cache.table.clone()
    table[0, 1], table[1, 0] = cache.num_pages + 5, -3
    a = Attn(lens, cache, 4, seed=3, table=table)
    for i in range(2):
        cache.values[i][0] = torch.cat([cache.values[i][0][:16], cache.values[i][0][32:]])
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
    a.check(lens=[48, 0])


def test_captured():
    lens = [300, 1000, 5]
    cache = bc.BlockCache(lens, 32, 16, 8, 128, "head", seed=9)
    a = Attn(lens, cache, 32, seed=3)
    a.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        binding.gemv_attn_decode(a.args, a.rec)
    torch.cuda.synchronize()
    for _ in range(3):
        a.guard[1:-1].fill_(-777.0)
        graph.replay()
        torch.cuda.synchronize()
        a.check()
