"""What the calls refuse of a cache with a scale for each block of tokens and
head, and of rows to be read back, before anything is launched."""
import math

import pytest

from memory_bound_decode_gb300 import binding, build_lib
from tests import blocks_cache as bc
from tests.test_attn_cpu import A16, ALIGN, INVALID, attn, cache, rope

ROOM = 1 << 40
BLOCK = dict(kind=binding.GEMV_CACHE_FP8_BLOCK, k_block_scale=A16, v_block_scale=A16, block_tokens=8,
             scale_page_stride=4, scale_block_stride=2, scale_head_stride=1)


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def read(**over):
    f = dict(table=A16, table_width=4, table_stride=4, row_start=A16, requests=3, rows=10, k_out=A16, v_out=A16,
             k_out_stride=128, v_out_stride=128)
    f.update(over)
    return binding.cache_read_args(**f)


@pytest.mark.parametrize("over,status", [
    (dict(k_block_scale=0), INVALID), (dict(v_block_scale=None), INVALID), (dict(k_scale=A16), INVALID),
    (dict(v_scale=A16), INVALID), (dict(block_tokens=0), INVALID), (dict(block_tokens=-8), INVALID),
    (dict(block_tokens=5), INVALID), (dict(block_tokens=32), INVALID), (dict(page_size=128, block_tokens=128), INVALID),
    (dict(scale_page_stride=0), INVALID), (dict(scale_block_stride=0), INVALID), (dict(scale_head_stride=0), INVALID),
    (dict(scale_page_stride=-1), INVALID), (dict(scale_page_stride=1 << 60), INVALID),
    (dict(scale_page_stride=1 << 58), INVALID), (dict(scale_head_stride=1 << 62), INVALID),
    (dict(scale_block_stride=(1 << 63) - 1), INVALID), (dict(head_dim=72), INVALID), (dict(kind=2), INVALID),
    (dict(kind=4), INVALID), (dict(k_block_scale=A16 + 2), ALIGN), (dict(v_block_scale=A16 + 1), ALIGN),
    (dict(slot_stride=136), ALIGN), (dict(k=A16 + 8), ALIGN),
])
def test_cache_refusals(over, status):
    c = cache(**{**BLOCK, **over})
    assert binding.gemv_attn_decode(attn(workspace_bytes=ROOM), c, 0, check=False) == status
    assert binding.gemv_cache_read(read(), c, 0, check=False) == status
    if "head_dim" not in over:
        assert binding.gemv_rope_append(rope(v=A16, v_stride=128, slots=A16), c, 0, check=False) == status


def test_fields_of_other_kinds():
    """A cache without scales for blocks may hold anything where their fields are: a call gets as far as it did."""
    junk = dict(k_block_scale=A16 + 1, block_tokens=-3, scale_page_stride=-1)
    for kind in (binding.GEMV_CACHE_BF16, binding.GEMV_CACHE_FP8):
        empty = attn(requests=0, workspace_bytes=ROOM)
        assert binding.gemv_attn_decode(empty, cache(kind=kind, **junk), 0) == binding.GEMV_OK
        assert binding.gemv_cache_read(read(requests=0), cache(kind=kind, **junk), 0) == binding.GEMV_OK


def test_one_page_one_block_one_head():
    """A dimension of one entry needs no stride."""
    c = cache(**{**BLOCK, "num_pages": 1, "block_tokens": 16, "kv_heads": 1, "scale_page_stride": 0,
                 "scale_block_stride": 0, "scale_head_stride": 0})
    assert binding.gemv_cache_read(read(rows=0), c, 0) == binding.GEMV_OK


@pytest.mark.parametrize("over,status", [
    (dict(table=0), INVALID), (dict(row_start=None), INVALID), (dict(k_out=None, v_out=0), INVALID),
    (dict(requests=-1), INVALID), (dict(requests=(1 << 30) + 1), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), INVALID), (dict(table_width=0), INVALID), (dict(table_stride=3), INVALID),
    (dict(table_stride=(1 << 31) + 1), INVALID), (dict(table_width=1 << 27, table_stride=1 << 27), INVALID),
    (dict(k_out_stride=120), INVALID), (dict(v_out_stride=0), INVALID), (dict(k_out_stride=(1 << 31) + 8), INVALID),
    (dict(row_type=2), INVALID), (dict(row_type=-1), INVALID), (dict(k_out=A16 + 8), ALIGN), (dict(v_out=A16 + 2), ALIGN),
    (dict(k_out_stride=132), ALIGN), (dict(row_type=0, v_out_stride=130), ALIGN), (dict(table=A16 + 2), ALIGN),
    (dict(begin=A16 + 1), ALIGN), (dict(row_start=A16 + 3), ALIGN),
])
def test_read_refusals(over, status):
    assert binding.gemv_cache_read(read(**over), cache(**BLOCK), 0, check=False) == status


def test_read_of_nothing():
    assert binding.gemv_cache_read(read(requests=0), cache(**BLOCK), 0) == binding.GEMV_OK
    assert binding.gemv_cache_read(read(rows=0, k_out=None, k_out_stride=0), cache(), 0) == binding.GEMV_OK
    assert binding.gemv_rope_append(rope(v=A16, v_stride=128, slots=A16, tokens=0), cache(**BLOCK), 0) == binding.GEMV_OK


@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (16, 128), (16, 256)])
def test_workspace_is_the_fp8_caches(heads, dim):
    of = [binding.gemv_attn_query(16, heads, dim, k, 152) for k in (binding.GEMV_CACHE_FP8, binding.GEMV_CACHE_FP8_BLOCK)]
    assert of[0] == of[1]


def test_the_definition_of_a_scale():
    """need() of the helpers against a search over the powers of two."""
    for a in (0.0, 1e-45, 1e-9, 448 * 2.0 ** -30, 448 * 2.0 ** -30 * (1 + 2 ** -23), 1.0, 447.99, 448.0, 448.001, 3e38):
        p = bc.FLOOR
        while p * 448 < a:
            p *= 2
        assert bc.need(a) == p and math.log2(p) == round(math.log2(p))
