"""gemv_attn_decode against the definition in 64 bits, through the C ABI."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au

pytestmark = pytest.mark.gpu


def run(lens, q_heads, heads, dim, page, kind="bf16", layout="token", **kw):
    extra = kw.pop("extra", 0)
    cache = au.Cache(lens, page, heads, dim, kind, layout, seed=len(lens) + page + dim, extra=extra)
    a = au.Attn(lens, cache, q_heads, **kw)
    a.run()
    torch.cuda.synchronize()
    a.check()
    assert binding.gemv_device_status() == 0
    return a


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 0, 127, 128, 129]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 128])
def test_edges_of_length_and_page(kind, layout, page):
    run(EDGES, 8, 2, 64, page, kind, layout)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_sizes(kind, dim):
    run([5, 300, 0, 64, 1000], 8, 2, dim, 16, kind)


@pytest.mark.parametrize("dim", [8, 72, 120, 248])
def test_head_sizes_of_eight(dim):
    run([5, 300, 0, 64], 4, 2, dim, 16)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 5, 8, 9, 16, 17, 32, 33, 71])
def test_groups(kind, dim, group):
    run([1, 100, 513], group * 2, 2, dim, 16, kind, "head")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [40], [5000], [20011], [20000] * 3, list(range(300)), [1] * 700])
def test_splits(kind, lens):
    """One row over many CTAs, many rows in one CTA, more requests than threads."""
    run(lens, 4, 1, 128, 32, kind, "head")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
def test_window(kind, window):
    run([0, 1, 2, 16, 17, 99, 100, 101, 116, 117, 3001], 8, 2, 128, 24, kind, window=window)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_softcap_and_scale(kind):
    run([1, 77, 1024], 8, 2, 64, 16, kind, softcap=5.0)
    run([1, 77, 1024], 8, 2, 64, 16, kind, softcap=30.0, window=50, scale=0.5)
    run([1, 77, 1024], 8, 2, 64, 16, kind, scale=-0.25)
    run([1, 77, 1024], 8, 2, 64, 16, kind, scale=0.0)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_strides(kind):
    """Pages inside a larger pool, rows of q and out apart, no lse."""
    run([40, 0, 333], 8, 2, 80, 16, kind, extra=16 * 5, pad=12, lse=False)


def test_queries_by_token_start_and_skipped_requests():
    """Request r's query is the last of its new tokens; requests without any, or of negative length, are left."""
    lens = [50, 7, 300, 0, 64, -1, 20]
    starts = [0, 3, 3, 4, 6, 6, 7, 8]
    cache = au.Cache(lens, 16, 2, 64, seed=3)
    a = au.Attn(lens, cache, 8, token_start=starts, rows=10)
    a.run()
    torch.cuda.synchronize()
    a.check()
    a = au.Attn(lens, cache, 8)     # a row per request: the negative length's is left
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_token_start_out_of_range_is_skipped():
    lens = [50, 60]
    cache = au.Cache(lens, 16, 2, 64, seed=3)
    a = au.Attn(lens, cache, 8, token_start=[0, 1, 9], rows=2)
    binding.gemv_device_status()
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
    mark = float(torch.tensor(-777.0).bfloat16())
    assert (a.out[1].float() == mark).all() and (a.out[0].float() != mark).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_pages_outside_the_pool_count_as_masked(kind):
    lens = [64, 40]
    cache = au.Cache(lens, 16, 2, 64, kind, seed=5)
    bad = cache.table.clone()
    bad[0, 1], bad[1, :] = cache.num_pages, -1
    a = au.Attn(lens, cache, 8, table=bad)
    binding.gemv_device_status()
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
    assert (a.out[1].float() == 0).all() and (a.lse[1] == -math.inf).all()
    keep = [i for i in range(64) if not 16 <= i < 32]
    k, v = (cache.values[i][0][keep] for i in range(2))
    out, z, mass, size = au.attend(a.q[0].cpu().view(8, 64), k, v, a.scale)
    tol, tol_z = au.attn_bounds(out, z, mass, size, 64, 64, kind)
    assert ((a.out[0].double().cpu().view(8, 64) - out).abs() <= tol).all()
    assert ((a.lse[0].double().cpu() - z).abs() <= tol_z).all()


def test_length_past_the_table_is_cut():
    cache = au.Cache([48], 16, 2, 64, seed=5)
    a = au.Attn([100], cache, 8)
    binding.gemv_device_status()
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == binding.GEMV_STATUS_BAD_PAGE
    a.check(lens=[48])


def test_peaked_scores_and_late_maximum():
    """Scores that differ by far more than the exponent's range, the largest first or last."""
    n, D = 700, 64
    for where in (0, 350, n - 1):
        cache = au.Cache([n], 16, 1, D, seed=9)
        q = torch.zeros(1, 4, D, dtype=torch.bfloat16)
        q[..., 0] = 100.0
        vk = cache.view(0)
        for j in range(n):
            val = 60.0 if j == where else -float(j % 50)
            vk[int(cache.table[0, j // 16]), j % 16, 0, 0] = val
            cache.values[0][0][j, 0, 0] = float(torch.tensor(val).bfloat16())
        a = au.Attn([n], cache, 4, q=q.cuda(), scale=1.0)
        a.run()
        torch.cuda.synchronize()
        a.check()


def test_infinite_and_nan_keys():
    """A NaN key makes its heads NaN, as the definition does; other requests are untouched."""
    lens = [40, 40]
    cache = au.Cache(lens, 16, 2, 64, seed=5)
    cache.view(0)[int(cache.table[0, 1]), 3, 1, 5] = float("nan")
    a = au.Attn(lens, cache, 8)
    a.run()
    torch.cuda.synchronize()
    o = a.out.float().view(2, 8, 64)
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(a.lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all()
    cache = au.Cache(lens, 16, 2, 64, seed=5)
    a = au.Attn(lens, cache, 8)
    cache.view(0)[int(cache.table[0, 1]), 3, 1, 5] = -math.inf * torch.sign(a.q[0, 4 * 64 + 5]).item()
    a.run()
    torch.cuda.synchronize()
    o = a.out.float().view(2, 8, 64)
    assert torch.isfinite(o[0, 4]).all()      # score -inf: that token has no weight


def test_same_bits_every_time_and_workspace_left_ready():
    lens = [9000, 3, 0, 4097, 811]
    cache = au.Cache(lens, 16, 2, 128, seed=2)
    a = au.Attn(lens, cache, 16)
    outs = []
    for _ in range(4):
        a.run()
        torch.cuda.synchronize()
        outs.append((a.out.clone(), a.lse.clone()))
    for o, z in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0][0].view(torch.int16)) and torch.equal(z, outs[0][1])
    a.check()
    assert (a.ws[:4096] == 0).all()
    other = au.Cache([5000, 200], 24, 1, 64, seed=4)      # another shape on the same workspace
    b = au.Attn([5000, 200], other, 4, workspace=a.ws)
    b.run()
    torch.cuda.synchronize()
    b.check()


def test_two_streams_with_a_workspace_each():
    jobs = []
    for i in range(4):
        lens = [3000 + 17 * i, 5, 900]
        cache = au.Cache(lens, 16, 2, 64, seed=i)
        jobs.append((au.Attn(lens, cache, 8, seed=i), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in jobs:
            a.run(s)
    torch.cuda.synchronize()
    for a, _ in jobs:
        a.check()


def test_captured_and_replayed_with_new_lengths():
    lens = [700, 3, 64, 1]
    cache = au.Cache(lens, 16, 2, 64, seed=8)
    a = au.Attn(lens, cache, 8)
    a.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for new in ([700, 3, 64, 1], [1, 0, 33, 0], [699, 2, 50, 1]):
        a.lens_t.copy_(torch.tensor(new, dtype=torch.int32))
        a.guard.fill_(-777.0)
        a.lse.fill_(-777.0)
        graph.replay()
        torch.cuda.synchronize()
        a.check(lens=new)


def test_offsets_past_32_bits():
    """Pages that begin past 2^32 bytes, and past 2^31 elements of the pool."""
    page, heads, dim = 16, 2, 64
    stride = 1 << 27                              # elements from page to page: 20 pages, 5.4 GB
    n, pages = 300, 20
    pool = torch.empty(pages * stride, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(pool, (pages, page, heads, dim), (stride, heads * dim, dim, 1))
    rows = au.randn(1, pages, page, heads, dim, dtype=torch.bfloat16)
    view.copy_(rows)
    small = au.Cache([n], page, heads, dim, seed=1)
    small.num_pages, small.page_stride, small.width = pages, stride, pages
    order = torch.arange(pages - 1, -1, -1, dtype=torch.int32)
    small.table = order[None].cuda()
    small.pools = [pool, pool]
    vals = rows.cpu().double()[order.long()].reshape(-1, heads, dim)[:n]
    small.values = [[vals], [vals]]
    a = au.Attn([n], small, 8)
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_no_requests():
    cache = au.Cache([4], 16, 2, 64)
    a = au.Attn([4], cache, 8)
    a.args.requests = 0
    a.run()
    torch.cuda.synchronize()
    mark = float(torch.tensor(-777.0).bfloat16())
    assert (a.guard.float() == mark).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", [2, 4, 6, 8, 12, 32])
def test_heads_in_teams(kind, heads):
    """KV heads that divide into blocks of 2, 4 or 8 (and not): rows in one piece, cut in two, cut in many."""
    run([5000, 0, 3, 900, 2047, 64, 1, 6500], 4 * heads, heads, 64, 16, kind, "head")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads, n, requests", [
    (8, 700, 1), (8, 1000, 1), (8, 2000, 1), (8, 9001, 1),      # one request: 1, 4, 8 and more CTAs a row
    (1, 30000, 1), (2, 30000, 1),                               # rows joined in two levels
    (8, 1000, 8), (8, 2001, 8), (8, 1999, 13), (4, 515, 38),    # a row per CTA, rows in two, no room for all rows
    (8, 600, 20), (1, 33, 256), (1, 33, 257),                   # more rows than CTAs; the last one counted, the first not
])
def test_rows_of_one_length(kind, heads, n, requests):
    run([n] * requests, 4 * heads, heads, 64, 32, kind, "token")


def test_rows_of_one_length_in_groups_of_sixteen_and_wide_heads():
    run([2500] * 3, 32, 2, 256, 24, "bf16", "head")
    run([2500] * 3, 64, 4, 128, 16, "bf16", "token")
    run([2500] * 3, 66, 2, 128, 16, "fp8", "token")             # 33 heads a group: two tiles of them, teams of 2


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_small_weights_beside_a_large_one(kind):
    """One token takes nearly all the weight and has v = 0, so that the output is made of the others' weights alone:
    2^-9 down to 2^-24 of its own."""
    n, D, heads, G = 40, 64, 1, 4
    cache = au.Cache([n], 16, heads, D, kind, seed=12)
    one = 0x38 if kind == "fp8" else 1.0                       # the E4M3 code of 1
    for which in range(2):
        view = cache.view(which)
        for j in range(n):
            at = view[int(cache.table[0, j // 16]), j % 16, 0]
            if which == 0:
                at[:] = 0                                      # k = (j's part of the score, 0, ..)
                cache.values[0][0][j, 0] = 0.0
                if j == 7:
                    at[0] = one
                    cache.values[0][0][j, 0, 0] = 1.0 if kind == "bf16" else float(cache.scales[0][0])
            elif j == 7:
                at[:] = 0
                cache.values[1][0][j, 0] = 0.0
    k0 = float(cache.values[0][0][7, 0, 0])
    q = torch.zeros(1, heads * G, D, dtype=torch.bfloat16)
    for h, drop in enumerate((9.0, 14.0, 17.5, 24.0)):          # the large weight is 2^drop of the others'
        q[0, h, 0] = drop * math.log(2.0) / k0
    a = au.Attn([n], cache, heads * G, q=q.cuda(), scale=1.0)
    a.run()
    torch.cuda.synchronize()
    a.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("drop", [10, 17, 24])
def test_small_queries_beside_a_large_one(kind, drop):
    """A column where q is large and every k is 0: the scores are made of columns 2^-drop of it, in full precision."""
    n, D = 50, 64
    cache = au.Cache([n], 16, 1, D, kind, seed=13)
    view = cache.view(0)
    for j in range(n):
        view[int(cache.table[0, j // 16]), j % 16, 0, 5] = 0
        cache.values[0][0][j, 0, 5] = 0.0
    q = (au.randn(3, 1, 4, D, device="cpu") * 2.0 ** -drop).bfloat16()
    q[..., 5] = 3.0
    a = au.Attn([n], cache, 4, q=q.cuda(), scale=0.25 * 2.0 ** drop)
    a.run()
    torch.cuda.synchronize()
    a.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("group, heads, dim", [(1024, 2, 256), (520, 4, 256), (1000, 1, 64)])
def test_many_head_tiles_and_one_team(kind, group, heads, dim):
    run([700, 3, 0, 2000], group * heads, heads, dim, 16, kind, "head")


@pytest.mark.parametrize("dim", [8, 24, 40, 56, 88, 104, 136, 200, 216, 232, 240, 248])
def test_head_sizes_cut_between_ctas(dim):
    """Items of a join are numbered through heads of dim / 4 columns."""
    run([9000], 7, 1, dim, 16)
    run([2100, 300], 62, 2, dim, 16)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("requests", [31, 32, 33, 255, 256, 257, 513])
def test_counts_of_requests(kind, requests):
    """Each warp, each CTA, or chunk after chunk sums the lengths up."""
    lens = [(i * 37) % 211 if i % 9 else 0 for i in range(requests)]
    lens[requests - 1] = 777
    starts = [0]
    for i in range(requests):
        starts.append(starts[-1] + (0 if i % 11 == 3 else 1 + i % 2))
    run(lens, 8, 2, 64, 16, kind, "token")
    run(lens, 8, 2, 64, 16, kind, "head", token_start=starts, rows=starts[-1] + 1, window=100)
