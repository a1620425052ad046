"""gemv_cache_read against the cache's values, rounded once: every row of a
request's tokens, every other element as it was."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au
from tests import blocks_cache as bc

pytestmark = pytest.mark.gpu
MARK = -777.0


def make(kind, lens, page, block, heads, dim, layout="token", seed=0, **more):
    if kind == "block":
        return bc.BlockCache(lens, page, block, heads, dim, layout, seed=seed, powers=seed % 2 == 0, **more)
    return au.Cache(lens, page, heads, dim, kind, layout, seed=seed, **more)


class Read:
    def __init__(self, cache, begin, count, row_type="bf16", pad=0, behind=0, table=None, use_begin=True):
        self.cache, self.begin, self.count = cache, begin, count
        self.total, R = sum(count), len(count)
        self.rows = self.total + behind
        W = cache.heads * cache.dim
        dt = torch.bfloat16 if row_type == "bf16" else torch.float32
        self.dt, self.W, self.stride = dt, W, W + pad
        self.out = [torch.full((self.rows + 2, self.stride), MARK, dtype=dt, device="cuda") for _ in range(2)]
        start = [0]
        for n in count:
            start.append(start[-1] + n)
        self.start = start
        i32 = dict(dtype=torch.int32, device="cuda")
        self.args = dict(table=cache.table if table is None else table, table_width=cache.width, table_stride=cache.width,
                         begin=torch.tensor(begin, **i32) if use_begin else None, row_start=torch.tensor(start, **i32),
                         requests=R, rows=self.rows, k_out=self.out[0][1:], v_out=self.out[1][1:],
                         k_out_stride=self.stride, v_out_stride=self.stride,
                         row_type=binding.GEMV_ROWS_BF16 if row_type == "bf16" else binding.GEMV_ROWS_F32)

    def run(self, stream=None, **over):
        self.rec = binding.cache_read_args(**{**self.args, **over})
        self.cache_rec = self.cache.record()
        binding.gemv_cache_read(self.rec, self.cache_rec, stream)

    def check(self, only=(0, 1), zeros=()):
        """`zeros`: rows that read as zeros."""
        torch.cuda.synchronize()
        mark = float(torch.tensor(MARK).to(self.dt))
        for i in range(2):
            got = self.out[i].cpu()
            if i not in only:
                assert (got.float() == mark).all()
                continue
            assert (got[0].float() == mark).all() and (got[1 + self.total:].float() == mark).all(), "a row without a token"
            assert (got[:, self.W:].float() == mark).all(), "write between rows"
            for r, n in enumerate(self.count):
                b = self.begin[r]
                want = self.cache.values[i][r][b:b + n].float().to(self.dt).reshape(n, self.W)
                have = got[1 + self.start[r]:1 + self.start[r + 1], :self.W].clone()
                for row in zeros:
                    if self.start[r] <= row < self.start[r + 1]:
                        want[row - self.start[r]] = 0
                assert torch.equal(have, want), (i, r)


@pytest.mark.parametrize("kind", ["block", "fp8", "bf16"])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("row_type", ["bf16", "f32"])
@pytest.mark.parametrize("page,block,heads,dim,lens", [
    (16, 16, 8, 128, [300]), (24, 8, 3, 80, [0, 5, 24, 77, 0, 0, 1]), (1, 1, 1, 64, [9, 3]), (64, 32, 2, 256, [130, 64, 63]),
    (8, 4, 16, 16, [1, 7, 8, 9, 250]), (128, 64, 5, 96, [1000, 2])])
def test_read(kind, layout, row_type, page, block, heads, dim, lens):
    c = make(kind, lens, page, block, heads, dim, layout, seed=page + dim, extra=16)
    begin = [n // 3 for n in lens]
    r = Read(c, begin, [n - b for n, b in zip(lens, begin)], row_type, pad=8, behind=3)
    r.run()
    r.check()
    r = Read(c, [0] * len(lens), lens, row_type, use_begin=False)
    r.run()
    r.check()
    assert binding.gemv_device_status() == 0


def test_one_of_the_two():
    c = make("block", [50, 20], 16, 8, 4, 64)
    r = Read(c, [0, 0], [50, 20])
    r.run(k_out=None, k_out_stride=0)
    r.check(only=(1,))
    r = Read(c, [0, 0], [50, 20])
    r.run(v_out=None)
    r.check(only=(0,))


def test_many_requests():
    """More requests than a CTA has threads, long stretches of empty ones among them."""
    lens = [(r * 7) % 5 if r % 3 else 0 for r in range(1500)] + [0] * 700 + [3, 0, 40] + [0] * 300
    c = make("block", lens, 8, 8, 2, 64, seed=2)
    r = Read(c, [0] * len(lens), lens, behind=40)
    r.run()
    r.check()


@pytest.mark.parametrize("requests", [255, 256, 257, 4096, 65536, 65537, 70001])
def test_numbers_of_requests(requests):
    """Numbers of requests on both sides of what one and two rounds of the search take; runs of requests without a row."""
    g = torch.Generator().manual_seed(requests)
    codes = torch.randint(0, 0x7F, (2, 512, 4, 1, 16), generator=g, dtype=torch.uint8).cuda()
    scales = torch.exp2(torch.randint(-6, 7, (2, 512, 2), generator=g).float()).cuda()
    table = torch.randint(0, 512, (requests, 1), generator=g, dtype=torch.int32).cuda()
    begin = torch.randint(0, 3, (requests,), generator=g, dtype=torch.int32).cuda()
    count = torch.randint(0, 3, (requests,), generator=g) * (torch.arange(requests) // 700 % 2)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])
    rows = max(1, int(start[-1]))
    out = [torch.full((rows, 16), MARK, device="cuda") for _ in range(2)]
    cache = binding.kv_cache(codes[0], codes[1], kind=binding.GEMV_CACHE_FP8_BLOCK, num_pages=512, page_size=4, kv_heads=1,
                             head_dim=16, page_stride=64, head_stride=16, slot_stride=16, block_tokens=2,
                             k_block_scale=scales[0], v_block_scale=scales[1], scale_page_stride=2, scale_block_stride=1,
                             scale_head_stride=1)
    start_t = start.to(torch.int32).cuda()
    binding.gemv_cache_read(binding.cache_read_args(
        table=table, table_width=1, table_stride=1, begin=begin, row_start=start_t, requests=requests, rows=rows,
        k_out=out[0], v_out=out[1], k_out_stride=16, v_out_stride=16, row_type=binding.GEMV_ROWS_F32), cache)
    torch.cuda.synchronize()
    of = torch.repeat_interleave(torch.arange(requests), count).cuda()
    tok = begin[of] + torch.arange(len(of)).cuda() - start.cuda()[of]
    ok = tok < 4                                   # (the others are past their row of the table: zeros, and the status bit)
    page, tok = table[of, 0].long(), tok.clamp(max=3)
    for i in range(2):
        want = codes[i][page, tok, 0].view(torch.float8_e4m3fn).float() * scales[i][page, tok // 2, None]
        want = torch.where(ok[:, None], want, torch.zeros_like(want))
        assert torch.equal(out[i][:len(of)], want)
    assert binding.gemv_device_status() == (0 if ok.all() else binding.GEMV_STATUS_BAD_PAGE)


def test_fewer_rows_than_tokens():
    """No row past `rows` is written."""
    c = make("block", [50, 20], 16, 8, 4, 64)
    r = Read(c, [0, 0], [50, 20])
    r.run(rows=33)
    torch.cuda.synchronize()
    assert (r.out[0][34:].float() == float(torch.tensor(MARK).bfloat16())).all()
    want = c.values[0][0][:33].float().bfloat16().reshape(33, -1)
    assert torch.equal(r.out[0][1:34].cpu(), want)


@pytest.mark.parametrize("kind", ["block", "bf16"])
def test_pages_outside_the_pool(kind):
    """Zeros, and the status bit; the other rows as they should be."""
    c = make(kind, [60, 20], 16, 16, 2, 64, seed=4)
    table = c.table.clone()
    table[0, 1], table[0, 3], table[1, 0] = -1, c.num_pages, 2 ** 31 - 1
    r = Read(c, [10, 0], [50, 20], table=table)
    binding.gemv_device_status(reset=True)
    r.run()
    zeros = [j - 10 for j in range(10, 60) if 16 <= j < 32 or 48 <= j] + [50 + j for j in range(16)]
    r.check(zeros=zeros)
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
    assert binding.gemv_device_status() == 0


def test_tokens_outside_the_table():
    c = make("block", [32], 16, 16, 2, 64, seed=4)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full((40, 128), MARK, dtype=torch.float32, device="cuda")
    args = binding.cache_read_args(table=c.table, table_width=c.width, table_stride=c.width,
                                   begin=torch.tensor([-4], **i32), row_start=torch.tensor([0, 40], **i32), requests=1,
                                   rows=40, k_out=out, k_out_stride=128, row_type=binding.GEMV_ROWS_F32)
    rec = c.record()
    binding.gemv_cache_read(args, rec)
    torch.cuda.synchronize()
    assert (out[:4] == 0).all() and (out[36:] == 0).all()
    assert torch.equal(out[4:36].cpu(), c.values[0][0].float().reshape(32, 128))
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE


def test_captured_and_on_another_stream():
    c = make("block", [100, 30], 16, 8, 8, 128)
    r = Read(c, [3, 0], [97, 30])
    r.run()
    r.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        binding.gemv_cache_read(r.rec, r.cache_rec)
    for o in r.out:
        o.fill_(MARK)
    graph.replay()
    r.check()
    for o in r.out:
        o.fill_(MARK)
    torch.cuda.synchronize()
    r.run(torch.cuda.Stream())
    r.check()
