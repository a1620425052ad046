"""gemv_attn_decode over a cache with a scale for each block on infinities and NaN that a request does see: what the definition
gives in 64 bits, with every other head, column and request held to the usual bounds."""
import math

import pytest
import torch

from tests import blocks_cache as bc
from tests.test_attn_blocks_gpu import Attn
from tests.test_attn_nonfinite_gpu import DIM, GROUP, HEADS, LENGTHS, check

pytestmark = pytest.mark.gpu


def make(lens, page, block, **kw):
    cache = bc.BlockCache(lens, page, block, HEADS, DIM, seed=len(lens))
    return Attn(lens, cache, HEADS * GROUP, **kw)


def put(a, which, r, j, h, d, code):
    """Code `code` of E4M3 for value d of token j, head h of request r's k (0) or v (1)."""
    c = a.cache
    page, place = int(c.host_table[r, j // c.page]), j % c.page
    c.codes_of(c.pools[which])[page, place, h, d] = code
    scale = float(c.scales_of(c.scales[which])[page, place // c.block, h])
    c.values[which][r][j, h, d] = float(torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double()) * scale


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])            # tensor copies, copies by every thread
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("lens", LENGTHS)
def test_nan_in_a_query(lens, softcap, page, block):
    a = make(lens, page, block, softcap=softcap)
    for r in range(0, len(lens), 2):
        a.q[r, 3 * DIM + 7] = math.nan
    seen = check(a)
    rows = sum(1 for r in range(0, len(lens), 2) if lens[r])
    assert seen["lse_nan"] == rows and seen["nan"] == rows * DIM


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_nan_in_keys(lens, page, block):
    a = make(lens, page, block)
    for r, n in enumerate(lens):
        if n:
            put(a, 0, r, (n - 1) * (r % 2), 1, 9, 0x7F)
    seen = check(a)
    assert seen["lse_nan"] == GROUP * sum(n > 0 for n in lens)


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_nan_in_values(lens, page, block):
    """NaN in its own column, whatever the weight of its token; the log-sum-exp is k's."""
    a = make(lens, page, block)
    for r, n in enumerate(lens):
        if n:
            put(a, 1, r, n // 2, 1, 9, 0xFF)
    seen = check(a)
    assert seen["nan"] == GROUP * sum(n > 0 for n in lens) and seen["lse_nan"] == 0


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_infinite_scores(lens, page, block):
    """A score of +inf: outputs NaN (inf / inf), the log-sum-exp +inf (NaN where a key's code is 0)."""
    a = make(lens, page, block)
    for r in range(0, len(lens), 2):
        a.q[r, 5 * DIM + 11] = math.inf
        if lens[r]:
            put(a, 0, r, lens[r] - 1, 1, 11, 0x38)
    seen = check(a)
    rows = sum(1 for r in range(0, len(lens), 2) if lens[r])
    assert seen["lse_inf"] + seen["lse_nan"] == rows


@pytest.mark.parametrize("page,block", [(16, 8), (7, 7)])
@pytest.mark.parametrize("lens", [[1], [40, 1, 0, 5], [3000]])
def test_every_score_minus_infinity(lens, page, block):
    a = make(lens, page, block)
    for r, n in enumerate(lens):
        a.q[r, 2 * DIM + 1] = math.inf
        for j in range(n):
            put(a, 0, r, j, 0, 1, 0xB8)
    seen = check(a)
    assert seen["none"] == sum(n > 0 for n in lens)
