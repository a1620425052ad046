"""The attention half of a decode step on a machine without a GPU: what the
calls refuse before anything is launched, the launch query, the frequencies."""
import math

import pytest

from memory_bound_decode_gb300 import binding, build_lib
from tests.blocks_ref import block_tables

A16 = 1 << 20   # a fake, 16-byte aligned address: never dereferenced by validation
SMS = 152
INVALID, ALIGN, UNSUPPORTED = binding.GEMV_ERR_INVALID, binding.GEMV_ERR_ALIGN, binding.GEMV_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def cache(**over):
    f = dict(k=A16, v=A16, num_pages=10, page_size=16, kv_heads=2, head_dim=64, page_stride=16 * 128, head_stride=64,
             slot_stride=128)
    f.update(over)
    return binding.kv_cache(f.pop("k"), f.pop("v"), **f)


def attn(**over):
    f = dict(q=A16, out=A16, lens=A16, requests=3, q_heads=8, q_stride=512, out_stride=512, table=A16, table_width=4,
             table_stride=4, scale=0.125, workspace=A16)
    f.update(over)
    return binding.attn_args(**f)


def rope(**over):
    f = dict(q=A16, k=A16, q_out=A16, positions=A16, freqs=A16, tokens=3, q_heads=8, kv_heads=2, head_dim=64,
             rot_dim=64, q_stride=512, k_stride=128, q_out_stride=512)
    f.update(over)
    return binding.rope_args(**f)


def tables(**over):
    f = dict(lens=A16, new_tokens=A16, requests=3, page_size=16, num_pages=10, table=A16, table_width=4, table_stride=4,
             free_pages=A16, free_cap=5, free_next=A16, max_tokens=8, slots=A16, positions=A16, token_start=A16,
             page_start=A16, new_lens=A16, status=A16, free_next_out=A16)
    f.update(over)
    return binding.block_tables_args(**f)


BAD_CACHE = [
    (dict(k=0), INVALID), (dict(v=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), INVALID),
    (dict(head_dim=264), INVALID), (dict(kind=2), INVALID), (dict(kind=1, head_dim=72), INVALID),
    (dict(num_pages=1 << 28), INVALID), (dict(page_stride=56), INVALID), (dict(slot_stride=0), INVALID),
    (dict(head_stride=-64), INVALID), (dict(page_stride=1 << 58), INVALID), (dict(k_scale=A16), INVALID),
    (dict(k=A16 + 8), ALIGN), (dict(v=A16 + 4), ALIGN), (dict(page_stride=16 * 128 + 4), ALIGN),
    (dict(kind=1, slot_stride=136), ALIGN), (dict(kind=1, v_scale=A16 + 2), ALIGN),
]


@pytest.mark.parametrize("over,status", BAD_CACHE)
def test_cache_refusals(over, status):
    assert binding.gemv_attn_decode(attn(), cache(**over), 0, check=False) == status
    d = over.get("head_dim", 64)
    r = rope(v=A16, v_stride=1024, slots=A16, head_dim=max(2, d), rot_dim=2, q_stride=4096, k_stride=1024,
             q_out_stride=4096)
    if "kv_heads" in over or d < 2 or d > 256:
        return
    assert binding.gemv_rope_append(r, cache(**over), 0, check=False) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(lens=0), INVALID), (dict(table=0), INVALID),
    (dict(workspace=0), INVALID), (dict(requests=-1), INVALID), (dict(q_heads=0), INVALID), (dict(q_heads=7), INVALID),
    (dict(q_stride=508), INVALID), (dict(out_stride=0), INVALID), (dict(table_width=0), INVALID),
    (dict(table_stride=3), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=math.inf), INVALID), (dict(window=-1), INVALID),
    (dict(token_start=A16, rows=-1), INVALID), (dict(q_stride=514), ALIGN), (dict(out_stride=513), ALIGN),
    (dict(q=A16 + 4), ALIGN), (dict(out=A16 + 2), ALIGN), (dict(lse=A16 + 2), ALIGN), (dict(lens=A16 + 1), ALIGN),
    (dict(table=A16 + 2), ALIGN), (dict(workspace=A16 + 8), ALIGN), (dict(token_start=A16 + 2), ALIGN),
    (dict(q_heads=2050, q_stride=1 << 18, out_stride=1 << 18), UNSUPPORTED),
])
def test_attention_refusals(over, status):
    assert binding.gemv_attn_decode(attn(**over), cache(), 0, check=False) == status
    assert binding.lib().gemv_attn_decode(None, None, None) == INVALID


def test_nothing_to_do():
    assert binding.gemv_attn_decode(attn(requests=0), cache(), 0) == 0
    assert binding.gemv_rope(rope(tokens=0, k_out=A16, k_out_stride=128), 0) == 0
    assert binding.gemv_rope_append(rope(tokens=0, v=A16, v_stride=128, slots=A16), cache(), 0) == 0


@pytest.mark.parametrize("over,status", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(q_out=0), INVALID), (dict(positions=0), INVALID),
    (dict(freqs=0), INVALID), (dict(tokens=-1), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(head_dim=63), INVALID), (dict(head_dim=258, rot_dim=2), INVALID), (dict(rot_dim=0), INVALID),
    (dict(rot_dim=7), INVALID), (dict(rot_dim=66), INVALID), (dict(rows=2), INVALID), (dict(pairs=2), INVALID),
    (dict(axes=0), INVALID), (dict(axes=9, pair_axis=A16, axis_stride=3), INVALID), (dict(axes=2, axis_stride=3), INVALID),
    (dict(axes=2, pair_axis=A16, axis_stride=2), INVALID), (dict(q_stride=511), INVALID), (dict(k_stride=127), INVALID),
    (dict(q_out_stride=511), INVALID), (dict(q_stride=1 << 41), INVALID), (dict(q=A16 + 2), ALIGN),
    (dict(rows=1, k=A16 + 1), ALIGN), (dict(q_out=A16 + 1), ALIGN), (dict(positions=A16 + 2), ALIGN),
    (dict(freqs=A16 + 4), ALIGN),
])
def test_rope_refusals(over, status):
    assert binding.gemv_rope(rope(k_out=A16, k_out_stride=128, **over), 0, check=False) == status
    assert binding.gemv_rope_append(rope(v=A16, v_stride=128, slots=A16, **over), cache(), 0, check=False) == status


def test_rope_forms_refuse_each_others_arguments():
    ok = dict(k_out=A16, k_out_stride=128)
    for bad, status in [(dict(), INVALID), (dict(ok, v=A16, v_stride=128), INVALID), (dict(ok, slots=A16), INVALID),
                        (dict(k_out=A16, k_out_stride=127), INVALID), (dict(k_out=A16 + 1, k_out_stride=128), ALIGN)]:
        assert binding.gemv_rope(rope(**bad), 0, check=False) == status
    ok = dict(v=A16, v_stride=128, slots=A16)
    for bad, status in [(dict(), INVALID), (dict(v=A16, v_stride=128), INVALID), (dict(ok, k_out=A16), INVALID),
                        (dict(ok, v_stride=127), INVALID), (dict(ok, slots=A16 + 2), ALIGN),
                        (dict(ok, kv_heads=1), INVALID), (dict(ok, head_dim=32, rot_dim=32), INVALID)]:
        assert binding.gemv_rope_append(rope(**bad), cache(), 0, check=False) == status


@pytest.mark.parametrize("over,status", [
    (dict(lens=0), INVALID), (dict(status=0), INVALID), (dict(free_next=0), INVALID), (dict(requests=0), INVALID),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(table_width=0), INVALID),
    (dict(free_cap=-1), INVALID), (dict(free_pages=0), INVALID), (dict(num_pages=1 << 28), INVALID),
    (dict(table_width=1 << 28, table_stride=1 << 28), INVALID), (dict(max_tokens=0), INVALID),
    (dict(max_tokens=1 << 31), INVALID), (dict(table_stride=3), INVALID), (dict(slots=A16 + 2), ALIGN),
    (dict(table=A16 + 1), ALIGN), (dict(free_next_out=A16 + 2), ALIGN),
])
def test_block_tables_refusals(over, status):
    assert binding.gemv_block_tables(tables(**over), 0, check=False) == status
    assert binding.lib().gemv_block_tables(None, None) == INVALID


@pytest.mark.parametrize("q_heads,kv_heads,dim,tile,tiles,dim_tile", [
    (32, 8, 128, 8, 1, 128), (8, 8, 64, 8, 1, 64), (32, 2, 128, 16, 1, 128), (32, 1, 80, 32, 1, 128),
    (71, 1, 64, 32, 3, 64), (64, 2, 256, 16, 2, 256), (32, 2, 136, 16, 1, 256),
])
def test_attention_query(q_heads, kv_heads, dim, tile, tiles, dim_tile):
    i = binding.gemv_attn_query(q_heads, kv_heads, dim, binding.GEMV_CACHE_BF16, SMS)
    assert (i["head_tile"], i["head_tiles"], i["dim_tile"]) == (tile, tiles, dim_tile)
    assert i["grid"] % tiles == 0 and i["grid"] <= SMS
    assert i["head_tile"] * tiles >= q_heads // kv_heads
    # two pieces a CTA and one a warp: outputs, maxima and sums
    assert i["workspace_bytes"] == 4096 + i["grid"] * (2 + i["warps_per_cta"]) * tile * (dim_tile + 2) * 4


@pytest.mark.parametrize("args", [(0, 1, 64, 0, SMS), (8, 0, 64, 0, SMS), (7, 2, 64, 0, SMS), (8, 2, 60, 0, SMS),
                                  (8, 2, 264, 0, SMS), (8, 2, 72, 1, SMS), (8, 2, 64, 2, SMS), (8, 2, 64, 0, 0)])
def test_attention_query_refusals(args):
    with pytest.raises(binding.GemvError) as e:
        binding.gemv_attn_query(*args)
    assert e.value.status == INVALID


def test_freqs():
    """inv_freq / (2 pi) modulo a turn, in units of 2^-64."""
    inv = [1.0, 0.5, 10000.0 ** -0.75, 2 * math.pi, 7.0, -1.0, 0.0]
    for f, got in zip(inv, binding.gemv_rope_freqs(inv)):
        turns = (got % (1 << 64)) / 2.0 ** 64
        want = (f / (2 * math.pi)) % 1.0
        # double arithmetic: a few units of 2^-53 of the turns before the whole ones go
        assert min(abs(turns - want), 1 - abs(turns - want)) <= 2.0 ** -50
    for bad in ([], [math.nan], [1.0, math.inf]):
        with pytest.raises(binding.GemvError):
            binding.gemv_rope_freqs(bad)


def test_block_tables_definition():
    """The reference the GPU tests use, on a case worked by hand."""
    table = [[4, -1, -1], [-1, -1, -1], [6, 7, -1]]
    got = block_tables([3, 0, 8], [2, 0, 1], table, 4, 3, 10, [9, 1, 2], 1, 5)
    assert got == dict(slots=[19, 4, 8, -1, -1], positions=[3, 4, 8, 0, 0], token_start=[0, 2, 2, 3],
                       page_start=[1, 2, 2], new_lens=[5, 0, 9], status=[0, 0, 0], free_next=3,
                       table=[[4, 1, -1], [-1, -1, -1], [6, 7, 2]])


def test_attention_workload_is_described():
    import bench
    assert bench.describe("attn_step:B16:L4096") == ("attn", None, 4096, 16)
    assert bench.describe("f8:attn_step:B1:L100") == ("attn", None, 100, 1)
    with pytest.raises(SystemExit):
        bench.describe("attn_step:B16")


@pytest.mark.parametrize("over", [
    dict(requests=1024, table_width=1 << 20, table_stride=1 << 20),      # 1024 * 2 * (2^20 + 2) slices of 16 tokens
    dict(requests=(1 << 31) - 1),                                        # 2 * (4 + 2) each
])
def test_more_slices_than_the_list_holds(over):
    with pytest.raises(binding.GemvError) as e:
        binding.gemv_attn_decode(attn(**over), cache())
    assert e.value.status == UNSUPPORTED
