"""The operators of a cache with a scale for each block as they are used
together: prompts written, decode steps that append to their blocks and attend
over them, captured and replayed, and the cache read back; and the attention
half of a step over it. Each stage is held to 64 bits on what the stage before
it really left."""
import pytest
import torch

from memory_bound_decode_gb300 import binding, workloads
from tests import attn_util as au
from tests import blocks_cache as bc
from tests.test_attn_blocks_gpu import MORE
from tests.test_append_blocks_gpu import check_k, same_bits

pytestmark = pytest.mark.gpu

TINY = dict(layers=2, hidden=512, intermediate=512, vocab=64, q_rows=512, kv_rows=256)


class Layer:
    """What the helpers of a BlockCache need of one layer of an AttentionStep."""

    def __init__(self, step, d):
        self.page = self.block = step.page_size
        self.heads, self.dim, self.num_pages = step.kv_heads, step.head_dim, step.num_pages
        self.slot_stride, self.head_stride = self.heads * self.dim, self.dim
        self.page_stride = self.page * self.heads * self.dim
        self.scale_page_stride, self.scale_block_stride, self.scale_head_stride = self.heads, self.heads, 1
        self.pools, self.scales = [d[n].view(torch.uint8).view(-1) for n in ("k", "v")], d["scales"]

    codes_of, scales_of, host = bc.BlockCache.codes_of, bc.BlockCache.scales_of, bc.BlockCache.host

    def values(self, which, slots):
        codes, scales = self.host()[which]
        c, s = self.codes_of(codes), self.scales_of(scales.view(-1))
        page, place = torch.tensor(slots) // self.page, torch.tensor(slots) % self.page
        return c[page, place].contiguous().view(torch.float8_e4m3fn).double() * s[page, place // self.block].double()[..., None]


def check(step, lens, before):
    """One step that has run, with `lens` tokens a request before it and the layers' caches as `before`."""
    B, D, P = step.batch, step.head_dim, step.page_size
    assert step.status.tolist() == [0] * B and step.new_lens.tolist() == [n + 1 for n in lens]
    table, slots = step.table.cpu(), step.slots.tolist()
    inv = torch.tensor(step.inv_freq, dtype=torch.float64)
    zero = torch.zeros(D // 2, dtype=torch.int32)
    for d, old in zip(step.layers, before):
        layer = Layer(step, d)
        after = layer.host()
        k, size = au.turn(d["y"][1].view(B, -1, D), step.positions[None], inv, zero, D, False)
        check_k(layer, old[0], after[0], k, size, slots)
        expect = [t.clone() for t in old[1]]
        bc.write(layer, *expect, d["y"][2].view(B, -1, D).cpu(), slots)
        assert torch.equal(after[1][0], expect[0]) and same_bits(after[1][1], expect[1])
        for r, n in enumerate(lens):
            at = [int(table[r, j // P]) * P + j % P for j in range(n + 1)]
            out, z, mass, sz = au.attend(d["q"][r].cpu().view(-1, D), layer.values(0, at), layer.values(1, at), D ** -0.5)
            tol, _ = au.attn_bounds(out, z, mass, sz, n + 1, D, "fp8")
            assert ((d["out"][r].double().cpu().view(-1, D) - out).abs() <= tol + 2 * MORE * mass).all(), r
    assert binding.gemv_device_status() == 0


def caches(step):
    torch.cuda.synchronize()
    return [Layer(step, d).host() for d in step.layers]


@pytest.mark.parametrize("advance", [False, True])
def test_step(advance):
    lens = [0, 15, 16, 200, 31]
    step = workloads.AttentionStep(TINY, lens, batch=5, cache="fp8_block", advance=advance, room=40, seed=3)
    before = caches(step)
    step.run()
    torch.cuda.synchronize()
    check(step, lens, before)
    step.capture()
    for i in range(4):
        before = caches(step)
        for d in step.layers:                      # other activations each step, some of them large: scales grow
            d["x"].mul_(2.5 if i % 2 else -0.5)
        step.launch()
        torch.cuda.synchronize()
        check(step, [n + 1 + i for n in lens] if advance else lens, before)


def test_prompts_then_steps_then_read_back():
    """Prompts of several requests in one call, single tokens one call each, then everything read back as rows: what was
    written, to half a step of its block's scale for each time it was rounded."""
    heads, dim, page, block = 4, 64, 32, 16
    prompts, steps = [45, 3, 130], 21
    lens = [n + steps for n in prompts]
    cache = bc.BlockCache(lens, page, block, heads, dim, "head", seed=3, fill=False)
    g = torch.Generator().manual_seed(5)
    rows = [[torch.randn(n, heads, dim, generator=g) * torch.exp2(torch.rand(n, 1, 1, generator=g) * 6 - 3) for n in lens]
            for _ in range(2)]
    freqs = binding.rope_freqs([0.0] * (dim // 2), device="cuda")   # no turn: k comes back as it was
    rec = cache.record()

    def append(spans):                             # (request, first, count)
        k, v = (torch.cat([rows[w][r][a:a + n] for r, a, n in spans]).reshape(-1, heads * dim).contiguous().cuda()
                for w in range(2))
        T = k.shape[0]
        slots = torch.tensor([s for span in spans for s in cache.slots_of(*span)], dtype=torch.int32).cuda()
        out = torch.empty(T, heads * dim, dtype=torch.bfloat16, device="cuda")
        args = binding.rope_args(q=k, k=k, v=v, q_out=out, positions=torch.zeros(T, dtype=torch.int32, device="cuda"),
                                 freqs=freqs, tokens=T, q_heads=heads, kv_heads=heads, head_dim=dim, rot_dim=dim,
                                 q_stride=heads * dim, k_stride=heads * dim, v_stride=heads * dim,
                                 q_out_stride=heads * dim, slots=slots)
        binding.gemv_rope_append(args, rec)
        torch.cuda.synchronize()
    append([(r, 0, n) for r, n in enumerate(prompts)])
    for i in range(steps):
        append([(r, n + i, 1) for r, n in enumerate(prompts)])
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    outs = [torch.empty(start[-1], heads * dim, device="cuda") for _ in range(2)]
    binding.gemv_cache_read(binding.cache_read_args(
        table=cache.table, table_width=cache.width, table_stride=cache.width,
        row_start=torch.tensor(start, dtype=torch.int32).cuda(), requests=3, rows=start[-1], k_out=outs[0], v_out=outs[1],
        k_out_stride=heads * dim, v_out_stride=heads * dim, row_type=binding.GEMV_ROWS_F32), rec)
    torch.cuda.synchronize()
    for which in range(2):
        scales = cache.scales_of(cache.scales[which].cpu())
        for r, n in enumerate(lens):
            got = outs[which][start[r]:start[r + 1]].cpu().view(n, heads, dim).double()
            want = rows[which][r].double()
            slot = torch.tensor(cache.slots_of(r, 0, n))
            s = scales[slot // page, slot % page // block].double()[..., None]
            # 2^-4 of the value as it was written, 2^-10 of a scale then and of each later one, which doubles at least.
            tol = torch.maximum(au.E4M3 * want.abs(), 2.0 ** -10 * s) + 2.0 ** -10 * s + (0 if which else 2.0 ** -20 * want.abs())
            assert ((got - want).abs() <= tol).all(), (which, r)
