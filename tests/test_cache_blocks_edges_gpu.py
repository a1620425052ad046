"""A cache with a scale for each block of tokens and head at its edges: pools
whose offsets pass 32 bits, positions at the ends of their type, queries turned
in place, calls at the same time, copies that never come."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding, build_lib
from tests import attn_util as au
from tests import blocks_cache as bc
from tests.test_append_blocks_gpu import same_bits
from tests.test_attn_blocks_gpu import Attn
from tests.test_rope_gpu import Case

pytestmark = pytest.mark.gpu


class Apart(bc.BlockCache):
    """The requests' pages and scales ``page_stride`` and ``scale_stride`` elements from each other."""

    def spread_out(self, page_stride, scale_stride):
        codes = [self.codes_of(p) for p in self.pools]
        scales = [self.scales_of(s) for s in self.scales]
        self.page_stride, self.scale_page_stride = page_stride, scale_stride
        self.pools = [torch.empty(self.num_pages * page_stride, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.empty(self.num_pages * scale_stride, device="cuda") for _ in range(2)]
        for i in range(2):
            self.codes_of(self.pools[i]).copy_(codes[i])
            self.scales_of(self.scales[i]).copy_(scales[i])


def test_offsets_past_32_bits():
    """Codes past 2^32 bytes and scales past 2^31 elements from the pool's start: the same bits as close together."""
    lens = [16 * 20, 16 * 25 - 3, 16 * 24]
    near = bc.BlockCache(lens, 16, 16, 2, 64, seed=3)
    far = Apart(lens, 16, 16, 2, 64, seed=3)
    far.spread_out(1 << 26, 1 << 25)
    assert far.num_pages > 64
    held = [n - 21 for n in lens]
    slots = [s for r, n in enumerate(lens) for s in near.slots_of(r, held[r], 21)]
    total = sum(lens)
    start = [0, lens[0], lens[0] + lens[1], total]
    results = []
    for cache in (near, far):
        c = Case(len(slots), 8, 2, 64, 64, seed=5)
        slots_t = torch.tensor(slots, dtype=torch.int32, device="cuda")
        binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots_t), cache.record())
        a = Attn(lens, cache, 8, seed=7)
        a.run()
        rows = [torch.full((total, 128), -777.0, device="cuda") for _ in range(2)]
        starts = torch.tensor(start, dtype=torch.int32, device="cuda")
        args = binding.cache_read_args(table=cache.table, table_width=cache.width, table_stride=cache.width,
                                       row_start=starts, requests=3, rows=total, k_out=rows[0], v_out=rows[1],
                                       k_out_stride=128, v_out_stride=128, row_type=binding.GEMV_ROWS_F32)
        binding.gemv_cache_read(args, cache.record())
        torch.cuda.synchronize()
        results.append([a.guard, a.lse, *rows] + [cache.scales_of(s).nan_to_num(-1.0) for s in cache.scales]
                       + [cache.codes_of(p) for p in cache.pools])
    for x, y in zip(*results):
        assert same_bits(x, y)
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("T", [1, 40])
def test_far_positions(T):
    """The angle is reduced exactly at the ends of a position's type, in k as in q: T = 1 by the form for single tokens."""
    pos = [2 ** 31 - 1, -(2 ** 31), 1 << 20, 1]
    cache = bc.BlockCache([48], 16, 16, 1, 64, seed=2, fill=False)
    for first in (pos if T == 1 else [None]):
        c = Case(T, 2, 1, 64, 64, seed=6)
        at = [first] if T == 1 else (pos * T)[:T]
        c.pos.copy_(torch.tensor([at], dtype=torch.int32))
        slots = torch.tensor(cache.slots_of(0, 0, T), dtype=torch.int32, device="cuda")
        binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots), cache.record())
        torch.cuda.synchronize()
        # 64 bits themselves are off by 2^31 * 2^-53 * a few in the angle at the far end: 2^-20 of |a| + |b|, as the turn is.
        turn = 2 * 2.0 ** -20
        want, size = c.turned(c.q, 2)
        tol = au.BF16 * want.abs() + (1 + au.BF16) * turn * size + 1e-38
        assert ((c.q_out.view(T, 2, 64).double().cpu() - want).abs() <= tol).all()
        want, size = c.turned(c.k, 1)
        codes, scales = cache.codes_of(cache.pools[0].cpu()), cache.scales_of(cache.scales[0].cpu())
        for t, s in enumerate(cache.slots_of(0, 0, T)):
            scale = scales[s // 16, 0].double()[:, None]
            got = codes[s // 16, s % 16].contiguous().view(torch.float8_e4m3fn).double() * scale
            tol = torch.maximum(au.E4M3 * want[t].abs(), 2.0 ** -10 * scale) + (1 + au.E4M3) * turn * size[t]
            assert ((got - want[t]).abs() <= tol).all(), t


@pytest.mark.parametrize("T", [3, 500])
def test_queries_in_place(T):
    """q_out may be q's rows, as in gemv_rope: rows of padding tokens stay as they were."""
    cache = bc.BlockCache([T], 16, 1, 2, 128, seed=2, fill=False)
    slots = cache.slots_of(0, 0, T)
    slots[T // 2] = -1
    slots_t = torch.tensor(slots, dtype=torch.int32, device="cuda")
    c = Case(T, 8, 2, 128, 128, f32=False, seed=4)
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots_t), cache.record())
    torch.cuda.synchronize()
    want = c.q_out.clone()
    want[T // 2] = c.q[T // 2]
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots_t, q_out=c.q), cache.record())
    torch.cuda.synchronize()
    assert same_bits(c.q, want)


def test_calls_at_the_same_time():
    """Two batches on two streams, each with a cache and a workspace of its own: as one after the other."""
    lens = [[300, 41, 0, 900], [77, 16, 512]]
    both = []
    for i in range(2):
        cache = bc.BlockCache(lens[i], 32, 16, 4, 128, seed=i)
        c = Case(len(lens[i]), 16, 4, 128, 128, seed=i + 2)
        slots = torch.tensor([cache.slots_of(r, n - 1, 1)[0] if n else -1 for r, n in enumerate(lens[i])],
                             dtype=torch.int32, device="cuda")
        a = Attn(lens[i], cache, 16, seed=i)
        total = sum(lens[i])
        rows = [torch.empty((total, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        start = torch.tensor([0] + torch.tensor(lens[i]).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        read = binding.cache_read_args(table=cache.table, table_width=cache.width, table_stride=cache.width,
                                       row_start=start, requests=len(lens[i]), rows=total, k_out=rows[0],
                                       v_out=rows[1], k_out_stride=512, v_out_stride=512)
        both.append((cache.record(), c.args(v=c.v, v_stride=c.sk, slots=slots), a, read, rows, (cache, c, slots, start)))

    def run(i, stream):
        rec, rope, a, read = both[i][:4]
        binding.gemv_rope_append(rope, rec, stream)
        binding.gemv_attn_decode(a.args, rec, stream)
        binding.gemv_cache_read(read, rec, stream)

    def results():
        torch.cuda.synchronize()
        out = [t.clone() for b in both for t in (b[2].guard, b[2].lse, *b[4], *b[5][0].pools)]
        for b in both:
            b[2].guard.fill_(-777.0)
            for t in b[4]:
                t.zero_()
        torch.cuda.synchronize()
        return out
    torch.cuda.synchronize()
    run(0, torch.cuda.current_stream().cuda_stream)
    run(1, torch.cuda.current_stream().cuda_stream)
    alone = results()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            run(i, streams[i].cuda_stream)
    for x, y in zip(alone, results()):
        assert same_bits(x, y)
    assert binding.gemv_device_status() == 0


@pytest.fixture(scope="module")
def drop_lib():
    return build_lib.build_debug_drop_x()


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])         # tensor copies, copies by every thread
@pytest.mark.parametrize("lens", [[1], [20] * 300, [300, 0, 40, 5], [2000, 9], [40000]])
def test_wait_runs_out_and_reports(drop_lib, page, block, lens):
    """A build that leaves copies out, as for the other caches: every row NaN, the status bit set, the workspace left as
    a call leaves it, and the regular library computes right after."""
    cache = bc.BlockCache(lens, page, block, 2, 64, seed=5)
    a = Attn(lens, cache, 8)
    with binding.use_library(drop_lib):
        a.run()
        torch.cuda.synchronize()
        assert binding.gemv_device_status() == binding.GEMV_STATUS_WAIT_TIMEOUT
        assert binding.gemv_device_status() == 0
    for r, n in enumerate(lens):
        if n:
            assert torch.isnan(a.out[r].float()).all() and torch.isnan(a.lse[r]).all(), r
        else:
            assert (a.out[r].float() == 0).all() and (a.lse[r] == -math.inf).all()
    assert (a.ws[:4096] == 0).all()
    a.run()
    torch.cuda.synchronize()
    a.check()
    assert binding.gemv_device_status() == 0
