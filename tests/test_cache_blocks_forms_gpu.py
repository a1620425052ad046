"""The cache write with a scale for each block in every form that its queries take, and calls at the same time that grow scales."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au
from tests import blocks_cache as bc
from tests.test_append_blocks_gpu import check, same_bits
from tests.test_attn_blocks_gpu import Attn
from tests.test_cache_read_gpu import Read
from tests.test_rope_gpu import Case

pytestmark = pytest.mark.gpu

# Of 152 SMs: one token a CTA, two from 608 tokens of so many heads on, four by asynchronous copies from 3,040 on.
TOKENS = [500, 700, 3100, 3503]
LAYOUTS = [(8, 128, 128, False, 1), (6, 256, 64, True, 3), (14, 80, 80, False, 1), (64, 16, 16, True, 1)]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("q_heads,dim,rot,interleaved,axes", LAYOUTS)
def test_queries_in_place(T, q_heads, dim, rot, interleaved, axes):
    """q_out may be q's rows, as in gemv_rope: rows of padding tokens stay as they were."""
    cache = bc.BlockCache([T], 16, 1, 2, dim, seed=2, fill=False)
    slots = cache.slots_of(0, 0, T)
    away = [0, 1, T // 2, T // 2 + 3, T - 1]
    for t in away:
        slots[t] = -1
    slots_t = torch.tensor(slots, dtype=torch.int32, device="cuda")
    c = Case(T, q_heads, 2, dim, rot, axes, interleaved, f32=False, seed=4)
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots_t), cache.record())
    torch.cuda.synchronize()
    want = c.q_out.clone()
    want[away] = c.q[away]
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots_t, q_out=c.q), cache.record())
    torch.cuda.synchronize()
    assert same_bits(c.q, want)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("q_heads,dim,rot,interleaved,axes", LAYOUTS)
def test_queries_are_those_of_the_other_caches(f32, T, q_heads, dim, rot, interleaved, axes):
    """q is turned the same way whatever the cache: the same bits."""
    c = Case(T, q_heads, 2, dim, rot, axes, interleaved, f32=f32, seed=T, far=100000)
    other = au.Cache([T], 16, 2, dim, "fp8", "token", seed=7)
    cache = bc.BlockCache([T], 16, 16, 2, dim, "token", seed=7)
    slots = torch.tensor(cache.slots_of(0, 0, T), dtype=torch.int32).cuda()
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots), other.record())
    torch.cuda.synchronize()
    want = c.q_out.clone()
    c.q_out.fill_(-777.0)
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots), cache.record())
    torch.cuda.synchronize()
    assert same_bits(want, c.q_out)


def test_calls_at_the_same_time():
    """Two batches on two streams, each with a cache and a workspace of its own. Pools and scales are as before the
    first call each time, and rows are large enough that begun blocks grow: codes, scales and queries as from one call after
    the other, and those as defined."""
    lens = [[300, 41, 0, 900, 64], [77, 16, 512]]
    both = []
    for i in range(2):
        cache = bc.BlockCache(lens[i], 32, 16, 4, 128, seed=i)
        c = Case(len(lens[i]) + 39, 16, 4, 128, 128, f32=bool(i), seed=i + 2)
        c.k, c.v = c.k * 64, c.v * 64
        slots = [cache.slots_of(r, n - 1, 1)[0] if n else -1 for r, n in enumerate(lens[i][:-1])]
        slots += cache.slots_of(len(lens[i]) - 1, lens[i][-1] - 40, 40)          # and a piece of 40 tokens
        slots_t = torch.tensor(slots, dtype=torch.int32, device="cuda")
        a = Attn(lens[i], cache, 16, seed=i)
        total = sum(lens[i])
        rows = [torch.empty((total, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        start = torch.tensor([0] + torch.tensor(lens[i]).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        read = binding.cache_read_args(table=cache.table, table_width=cache.width, table_stride=cache.width,
                                       row_start=start, requests=len(lens[i]), rows=total, k_out=rows[0],
                                       v_out=rows[1], k_out_stride=512, v_out_stride=512)
        both.append(dict(rec=cache.record(), rope=c.args(v=c.v, v_stride=c.sk, slots=slots_t), attn=a, read=read,
                         rows=rows, cache=cache, case=c, slots=slots, keep=(slots_t, start),
                         first=[t.clone() for t in cache.pools + cache.scales], before=cache.host()))

    def reset():
        torch.cuda.synchronize()
        for b in both:
            for t, x in zip(b["cache"].pools + b["cache"].scales, b["first"]):
                t.copy_(x)
            b["attn"].guard.fill_(-777.0)
            b["attn"].lse.fill_(-777.0)
            b["case"].q_out.fill_(-777.0)
            for t in b["rows"]:
                t.zero_()
        torch.cuda.synchronize()

    def run(b, stream):
        binding.gemv_rope_append(b["rope"], b["rec"], stream)
        binding.gemv_attn_decode(b["attn"].args, b["rec"], stream)
        binding.gemv_cache_read(b["read"], b["rec"], stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for b in both for t in (*b["cache"].pools, *b["cache"].scales, b["case"].q_out, b["attn"].guard,
                                                  b["attn"].lse, *b["rows"])]
    reset()
    for b in both:
        run(b, torch.cuda.current_stream().cuda_stream)
    alone = results()
    for b in both:
        check(b["case"], b["cache"], b["slots"], b["before"], b["cache"].host())
        grown = [(t > x).any() for t, x in zip(b["cache"].scales, b["first"][2:])]
        assert all(grown)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        reset()
        for b, s in zip(both, streams):
            run(b, s.cuda_stream)
        for x, y in zip(alone, results()):
            assert same_bits(x, y)
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("requests", [2, 3, 4, 8, 9, 10])
@pytest.mark.parametrize("length", [512, 513, 600, 1024, 1025])
def test_rows_of_one_length(requests, length):
    """Attention on both sides of the lengths and numbers of rows that are cut between CTAs."""
    cache = bc.BlockCache([length] * requests, 64, 32, 8, 64, "head", seed=length)
    a = Attn(cache=cache, lens=[length] * requests, q_heads=8, seed=3)
    for _ in range(2):
        a.guard.fill_(-777.0)
        a.run()
        torch.cuda.synchronize()
        a.check()


@pytest.mark.parametrize("row_type", ["bf16", "f32"])
@pytest.mark.parametrize("given", [(True, True), (False, False), (True, False), (False, True)])
def test_read_without_scales(row_type, given):
    """Rows of an FP8 cache whose scales per head are left out: 1."""
    c = au.Cache([70, 5], 16, 3, 80, "fp8", "token", seed=4)
    for i in range(2):
        if not given[i]:
            c.values[i] = [v / c.scales[i].double().cpu()[:, None] for v in c.values[i]]
            c.values[i] = [v.float().to(torch.float8_e4m3fn).double() for v in c.values[i]]      # the codes, as they are
            c.scales[i] = None
    r = Read(c, [3, 0], [67, 5], row_type, pad=8, behind=2)
    r.run()
    r.check()
    assert binding.gemv_device_status() == 0
