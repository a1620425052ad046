"""gemv_rope_append into a cache with a scale for each block of tokens and head:
v's codes and scales bit by bit against the definition, k's within the turn's
error, every other byte as it was."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au
from tests import blocks_cache as bc
from tests.test_rope_gpu import TURN, Case, close

pytestmark = pytest.mark.gpu


def tokens_of(cache, new):
    """Slots of the new tokens: `new` lists (request, first place, count), or None for a padding row."""
    slots = []
    for n in new:
        slots += [-1] if n is None else cache.slots_of(*n)
    return slots


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check_k(cache, before, after, want, size, slots):
    """The scale that `want` asks for (either one where its largest value is within the turn's error of a border), and
    codes within half a step of it; what no token touches as it was."""
    (old_codes, old_scales), (codes, scales) = before, after
    err = TURN * size
    a = want.abs().amax(-1)
    e = err.amax(-1)
    low = [t.clone() for t in before]
    bc.write(cache, *low, want.float(), slots, peak=(a - e).clamp(min=0))
    high = [t.clone() for t in before]
    bc.write(cache, *high, want.float(), slots, peak=a + e)
    got_s, low_s, high_s = (cache.scales_of(t) for t in (scales, low[1], high[1]))
    assert ((got_s == low_s) | (got_s == high_s) | (got_s.isnan() & low_s.isnan())).all()
    total = cache.num_pages * cache.page
    got_c, low_c, high_c = (cache.codes_of(t) for t in (codes, low[0], high[0]))
    new = torch.zeros(cache.num_pages, cache.page, dtype=torch.bool)
    for t, s in enumerate(slots):
        if not 0 <= s < total:
            continue
        page, place = s // cache.page, s % cache.page
        new[page, place] = True
        scale = got_s[page, place // cache.block].double()[:, None]
        val = got_c[page, place].contiguous().view(torch.float8_e4m3fn).double() * scale
        tol = torch.maximum(au.E4M3 * want[t].abs(), 2.0 ** -10 * scale) + (1 + au.E4M3) * err[t]
        assert ((val - want[t]).abs() <= tol).all(), (t, float(((val - want[t]).abs() / tol).max()))
    other = ~new[:, :, None, None]
    either = (got_c == low_c) | (got_c == high_c)
    assert (either | ~other).all(), "a byte that no new token has"
    behind = torch.ones_like(codes, dtype=torch.bool)
    cache.codes_of(behind)[:] = False
    assert (codes[behind] == old_codes[behind]).all(), "write behind a page"
    behind = torch.ones_like(scales, dtype=torch.bool)
    cache.scales_of(behind)[:] = False
    assert same_bits(scales[behind], old_scales[behind]), "write behind a page's scales"


def run_and_check(c, cache, slots):
    before = cache.host()
    slots_t = torch.tensor(slots, dtype=torch.int32).cuda()
    args = c.args(v=c.v, v_stride=c.sk, slots=slots_t)
    binding.gemv_rope_append(args, cache.record())
    torch.cuda.synchronize()
    after = cache.host()
    check(c, cache, slots, before, after)
    return args, after


def check(c, cache, slots, before, after):
    total = cache.num_pages * cache.page
    mark = float(torch.tensor(-777.0).bfloat16())
    live = torch.tensor([0 <= s < total for s in slots])
    want, size = c.turned(c.q, c.q_heads)
    got = c.q_out[:, :c.q_heads * c.dim].reshape(c.T, c.q_heads, c.dim)
    close(got[live.cuda()], want[live], size[live])
    assert (got[~live.cuda()].float() == mark).all() and (c.q_out[:, c.q_heads * c.dim:].float() == mark).all()
    v = c.v[:, :c.heads * c.dim].reshape(c.T, c.heads, c.dim).float().cpu()
    expect = [t.clone() for t in before[1]]
    bc.write(cache, *expect, v, slots)
    assert same_bits(after[1][1], expect[1]), "scales of v"
    assert torch.equal(after[1][0], expect[0]), "codes of v"
    k, size = c.turned(c.k, c.heads)
    check_k(cache, before[0], after[0], k, size, slots)


SHAPES = [
    # q_heads, heads, dim, rot, axes, interleaved, pad, offset
    (32, 8, 128, 128, 1, False, 0, 0), (4, 2, 256, 64, 3, False, 8, 0), (7, 7, 80, 80, 2, True, 0, 0),
    (3, 1, 96, 6, 1, False, 2, 0), (4, 2, 64, 64, 1, True, 0, 1), (2, 1, 16, 16, 1, False, 0, 0),
]
BATCHES = [
    # page, block, tokens held, new tokens: (request, first place, count) or None
    (16, 16, [7, 0, 16, 31], [(0, 7, 1), (1, 0, 1), (2, 16, 1), (3, 31, 1)]),
    (32, 16, [5, 40], [(0, 5, 90), None, None, (1, 40, 7)]),
    (64, 64, [3, 0], [(0, 3, 150), (1, 0, 64)]),
    (24, 24, [23, 24, 1], [None, (0, 23, 1), (1, 24, 24), (2, 1, 60)]),
    (24, 8, [3, 9], [(0, 3, 1), (1, 9, 33)]),
    (8, 1, [2, 0, 5], [(0, 2, 3), (1, 0, 1), (2, 5, 20)]),
    (1, 1, [4], [(0, 4, 5)]),
]


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_append(layout, f32, shape, batch):
    q_heads, heads, dim, rot, axes, inter, pad, offset = SHAPES[shape]
    page, block, held, new = BATCHES[batch]
    lens = list(held)
    for n in new:
        if n:
            lens[n[0]] = n[1] + n[2]
    cache = bc.BlockCache(lens, page, block, heads, dim, layout, seed=batch, extra=16)
    slots = tokens_of(cache, new)
    c = Case(len(slots), q_heads, heads, dim, rot, axes, inter, f32, seed=batch + 3, pad=pad, offset=offset)
    run_and_check(c, cache, slots)
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("requests,count,block", [(700, 1, 16), (1300, 1, 64), (5, 400, 16), (260, 5, 8)])
def test_many_tokens(f32, requests, count, block):
    """Windows of several tokens a warp: single tokens, long runs, and both borders."""
    lens = [(7 * r) % 90 for r in range(requests)]
    cache = bc.BlockCache([n + count for n in lens], 64, block, 2, 64, "head", seed=5)
    slots = tokens_of(cache, [(r, n, count) for r, n in enumerate(lens)])
    c = Case(len(slots), 4, 2, 64, 64, f32=f32, seed=requests)
    run_and_check(c, cache, slots)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("q_heads,heads,dim,rot,axes,inter", [
    (32, 2, 128, 128, 1, False), (20, 2, 256, 64, 3, False), (14, 1, 80, 80, 2, True), (64, 1, 16, 16, 1, False)])
def test_prompts(f32, q_heads, heads, dim, rot, axes, inter):
    """As many tokens as it takes for the queries to come by asynchronous copies; padding rows at odd places and at the end."""
    held, new = [7, 0, 16], [(0, 7, 1101), None, (1, 0, 1300), None, None, None, (2, 16, 903), None, None]
    cache = bc.BlockCache([h + n[2] for h, n in zip(held, [new[0], new[2], new[6]])], 32, 16, heads, dim, seed=dim, extra=16)
    slots = tokens_of(cache, new)
    run_and_check(Case(len(slots), q_heads, heads, dim, rot, axes, inter, f32, seed=8), cache, slots)


def test_slots_past_the_pool_and_negative():
    cache = bc.BlockCache([40, 8], 16, 8, 2, 64, "token", seed=2)
    total = cache.num_pages * cache.page
    slots = [total, -5] + cache.slots_of(0, 30, 3) + [2 ** 31 - 1, -(2 ** 31)] + cache.slots_of(1, 0, 1) + [-1]
    c = Case(len(slots), 4, 2, 64, 32, seed=8)
    run_and_check(c, cache, slots)


def test_no_token():
    cache = bc.BlockCache([40], 16, 8, 2, 64)
    before = cache.host()
    c = Case(3, 4, 2, 64, 64, seed=8)
    run_and_check(c, cache, [-1, -1, -1])
    for (a, b), (x, y) in zip(before, cache.host()):
        assert torch.equal(a, x) and same_bits(b, y)


@pytest.mark.parametrize("f32", [True, False])
def test_scales_at_their_borders(f32):
    """Largest values on both sides of 448 times a power of two, at the floor, zero, tiny and huge."""
    dt = torch.float32 if f32 else torch.bfloat16
    eps = torch.finfo(dt).eps
    tops = [448.0, 448.0 * (1 + eps), 448.0 * (1 - eps), 224.0, 1.0, 447.0, 512.0, 511.0, 0.0, 1e-30,
            448 * 2.0 ** -30, 448 * 2.0 ** -30 * (1 + eps), 448 * 2.0 ** -31, 2.0 ** -126, 3e38, 448 * 2.0 ** 119]
    lens = [1] * len(tops)
    cache = bc.BlockCache(lens, 8, 8, 2, 64, "token", seed=1)
    slots = tokens_of(cache, [(r, 0, 1) for r in range(len(tops))])
    c = Case(len(slots), 4, 2, 64, 64, f32=f32, seed=1)
    x = torch.randn(len(tops), 128, generator=torch.Generator().manual_seed(1)).clamp(-0.99, 0.99)
    for i, t in enumerate(tops):
        x[i] *= t
        x[i, 7] = x[i, 70] = t
        x[i, 9] = x[i, 80] = -t
    c.v = x.to(dt).cuda()
    c.k = torch.zeros_like(c.v)                   # every scale of k at the floor
    _, after = run_and_check(c, cache, slots)
    at = [cache.scales_of(after[1][1])[s // 8, 0, 0].item() for s in slots]
    assert at[:9] == [1.0, 2.0, 1.0, 0.5, 2.0 ** -8, 1.0, 2.0, 2.0, 2.0 ** -30] and at[9:13] == [2.0 ** -30] * 2 + [2.0 ** -29, 2.0 ** -30]


@pytest.mark.parametrize("old", [1.0, 2.0 ** -20, 2.0 ** -3, 0.75, 1.2345e-3, 2.0 ** 40])
def test_earlier_codes_move(old):
    """Every E4M3 code that a block may hold, under scales that grow by much, little, and not at all."""
    cache = bc.BlockCache([17, 32], 32, 16, 4, 64, "head", seed=3)
    c = Case(2, 4, 4, 64, 64, seed=3)
    slots = cache.slots_of(0, 15, 1) + cache.slots_of(1, 20, 1)
    for pool, scale in zip(cache.pools, cache.scales):
        scale.fill_(old)
        codes = torch.arange(pool.numel(), device="cuda").to(torch.uint8)
        pool.copy_(torch.where(codes & 0x7F == 0x7F, codes - 1, codes))       # but for NaN
    run_and_check(c, cache, slots)


@pytest.mark.parametrize("f32", [True, False])
def test_values_that_are_not_finite(f32):
    """Infinities take the largest code and do not count for the scale; NaN stays NaN, in its own place."""
    lens = [4, 20, 1, 3]
    cache = bc.BlockCache(lens, 16, 16, 2, 64, "token", seed=4)
    slots = tokens_of(cache, [(0, 0, 4), (1, 17, 3), (2, 0, 1), (3, 1, 2)])
    c = Case(len(slots), 4, 2, 64, 64, f32=f32, seed=4)
    c.v[1, 5], c.v[1, 66], c.v[5, 3], c.v[6, 127] = math.inf, -math.inf, math.nan, math.inf
    c.v[7] = math.nan                              # a head of nothing but NaN, and one of infinities
    c.v[8, :64] = -math.inf
    before = cache.host()
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=torch.tensor(slots, dtype=torch.int32).cuda()), cache.record())
    torch.cuda.synchronize()
    (_, _), (codes, scales) = cache.host()
    v = c.v.reshape(c.T, 2, 64).float().cpu()
    bc.write(cache, *before[1], v, slots)
    assert same_bits(scales, before[1][1])
    a, b = (t.view(torch.float8_e4m3fn).float() for t in (codes, before[1][0]))
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


def test_a_block_token_by_token():
    """A block filled by single calls: after each, its tokens stand for what was written. Where the scale grew, codes
    among the subnormals were rounded again, by half a step of 2^-9 of the scale then: with scales that double at
    least, 2^-10 (1 + 1/2 + 1/4 + ..) of the last one in all."""
    cache = bc.BlockCache([64], 32, 32, 2, 64, "token", seed=6, fill=False)
    g = torch.Generator().manual_seed(9)
    rows = torch.randn(64, 2, 64, generator=g) * torch.exp2(torch.rand(64, 2, 1, generator=g) * 12 - 6)
    for t in range(64):
        c = Case(1, 4, 2, 64, 64, seed=t)
        c.v = rows[t].reshape(1, 128).cuda()
        run_and_check(c, cache, cache.slots_of(0, t, 1))
        codes, scales = cache.host()[1]
        for j in range(t + 1):
            s = cache.slots_of(0, j, 1)[0]
            sc = cache.scales_of(scales)[s // 32, 0].double()[:, None]
            val = cache.codes_of(codes)[s // 32, s % 32].contiguous().view(torch.float8_e4m3fn).double() * sc
            want = rows[j].double()
            tol = torch.maximum(au.E4M3 * want.abs(), 2.0 ** -10 * sc) + 2.0 ** -10 * sc
            assert ((val - want).abs() <= tol).all(), (t, j)


def test_repeated_captured_and_elsewhere():
    """The same call again, replayed from a graph, and on another stream: the same bits."""
    cache = bc.BlockCache([37, 60, 9], 16, 16, 8, 128, "token", seed=11)
    slots = cache.slots_of(0, 20, 17) + cache.slots_of(1, 59, 1) + [-1] + cache.slots_of(2, 0, 9)
    c = Case(len(slots), 32, 8, 128, 128, seed=12)
    first = cache.host()
    args, after = run_and_check(c, cache, slots)
    rec = cache.record()

    def again():
        torch.cuda.synchronize()
        for (p, s), (x, y) in zip(after, cache.host()):
            assert torch.equal(p, x) and same_bits(s, y)
    binding.gemv_rope_append(args, rec)
    again()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        binding.gemv_rope_append(args, rec)
    for _ in range(2):
        for pool, scale, (p, s) in zip(cache.pools, cache.scales, first):
            pool.copy_(p)
            scale.copy_(s)
        graph.replay()
        again()
    for pool, scale, (p, s) in zip(cache.pools, cache.scales, first):
        pool.copy_(p)
        scale.copy_(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    binding.gemv_rope_append(args, rec, side)
    again()


def test_other_shapes_are_captured_after_a_first_call():
    """Kernels that no call has used yet may be used in a capture: the first call on the device has loaded them all."""
    cache = bc.BlockCache([2000, 70], 64, 64, 2, 256, "token", seed=13)
    recs = []
    for T, f32, offset in ((1900, True, 0), (1900, False, 0), (3, True, 1), (3, False, 1)):
        c = Case(T, 2, 2, 256, 256, f32=f32, seed=T, offset=offset)
        slots = cache.slots_of(0, 5, 1900) if T > 3 else cache.slots_of(1, 64, 3)
        slots_t = torch.tensor(slots, dtype=torch.int32).cuda()
        recs.append((c, slots, slots_t, c.args(v=c.v, v_stride=c.sk, slots=slots_t)))
    rec = cache.record()
    first = Case(1, 2, 2, 64, 64, seed=1)
    small = bc.BlockCache([1], 8, 8, 2, 64)
    binding.gemv_rope_append(first.args(v=first.v, v_stride=first.sk, slots=torch.tensor(small.slots_of(0, 0, 1),
                                        dtype=torch.int32).cuda()), small.record())
    for c, slots, _, args in recs:
        torch.cuda.synchronize()
        before = cache.host()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            binding.gemv_rope_append(args, rec)
        graph.replay()
        torch.cuda.synchronize()
        check(c, cache, slots, before, cache.host())


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,interleaved", [(3, False), (700, True)])
def test_queries_are_those_of_the_other_caches(f32, T, interleaved):
    """q is turned the same way whatever the cache: the same bits."""
    c = Case(T, 32, 2, 128, 128, f32=f32, interleaved=interleaved, seed=T, far=100000)
    other = au.Cache([T], 16, 2, 128, "fp8", "token", seed=7)
    cache = bc.BlockCache([T], 16, 16, 2, 128, "token", seed=7)
    slots = torch.tensor(cache.slots_of(0, 0, T), dtype=torch.int32).cuda()
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots), other.record())
    torch.cuda.synchronize()
    want = c.q_out.clone()
    c.q_out.fill_(-777.0)
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots), cache.record())
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), c.q_out.view(torch.int16))
