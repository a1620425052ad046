"""gemv_attn_decode on infinities and NaN that a request does see: what the definition gives in 64 bits, entry by
entry, with every other head, column and request held to the usual bounds."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, PAGE = 2, 4, 64, 16
# A token; rows within a warp's part, cut between warps, between CTAs, and joined in two levels; many rows a CTA.
LENGTHS = [[1], [40, 1, 0, 5], [777, 3], [9000], [40000], [20] * 300]


def make(lens, kind="bf16", **kw):
    cache = au.Cache(lens, PAGE, HEADS, DIM, kind, seed=len(lens))
    return au.Attn(lens, cache, HEADS * GROUP, **kw)


def put(a, which, r, j, h, d, value):
    """Value d of token j, head h of request r's k (0) or v (1): a BF16 value, or an E4M3 code."""
    c = a.cache
    c.view(which)[int(c.table[r, j // PAGE]), j % PAGE, h, d] = value
    if c.kind == "fp8":
        code = torch.tensor([value], dtype=torch.uint8).view(torch.float8_e4m3fn)
        value = float(code.double() * c.scales[which][h].double().cpu())
    c.values[which][r][j, h, d] = value


def check(a):
    """Against 64 bits: NaN where the definition has NaN, the same infinities, else within the bounds. A head whose
    scores are all -inf has no weight to share out: zeros."""
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == 0
    seen = dict(nan=0, inf=0, lse_nan=0, lse_inf=0, none=0)
    for r, n in enumerate(a.lens):
        if n == 0:
            continue
        k, v = (a.cache.values[i][r][:n] for i in range(2))
        out, z, mass, size = au.attend(a.q[r].cpu().view(-1, DIM), k, v, a.scale, a.softcap)
        tol, tol_z = au.attn_bounds(out, z, mass, size, n, DIM, a.cache.kind)
        out[z == -math.inf] = 0.0
        seen["none"] += int((z == -math.inf).sum())
        for got, want, bound, names in ((a.out[r].double().cpu().view(-1, DIM), out, tol, ("nan", "inf")),
                                        (a.lse[r].double().cpu(), z, tol_z, ("lse_nan", "lse_inf"))):
            nan, inf = want.isnan(), want.isinf()
            assert (got.isnan() == nan).all(), (r, n)
            assert (got[inf] == want[inf]).all(), (r, n)
            ok = want.isfinite()
            err = (got - want).abs()[ok]
            lim = torch.where(want == 0, bound.nan_to_num(0.0), bound)[ok]
            assert (err <= lim).all(), (r, n, float(err.max()))
            seen[names[0]] += int(nan.sum())
            seen[names[1]] += int((want == math.inf).sum())
    return seen


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("lens", LENGTHS)
def test_nan_in_a_query(lens, softcap, kind):
    """Every score of that head is NaN: so are its outputs and its lse."""
    a = make(lens, kind, softcap=softcap)
    for r in range(0, len(lens), 2):
        a.q[r, 3 * DIM + 7] = math.nan
    seen = check(a)
    rows = sum(1 for r in range(0, len(lens), 2) if lens[r])
    assert seen["lse_nan"] == rows and seen["nan"] == rows * DIM


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_nan_in_keys(lens, kind):
    """One NaN key is enough, whether it is the only token, the first or the last."""
    a = make(lens, kind)
    for r, n in enumerate(lens):
        if n:
            put(a, 0, r, (n - 1) * (r % 2), 1, 9, 0x7F if kind == "fp8" else math.nan)
    seen = check(a)
    assert seen["lse_nan"] == GROUP * sum(n > 0 for n in lens)


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_infinite_values(lens, where):
    """An infinite v makes its column infinite, of its own sign; both signs in a column make NaN."""
    a = make(lens)
    for r, n in enumerate(lens):
        if n == 0:
            continue
        j = dict(first=0, last=n - 1, middle=n // 2)[where]
        put(a, 1, r, j, 0, 3, math.inf)
        put(a, 1, r, j, 0, 60, -math.inf)
        put(a, 1, r, j, 1, 17, math.inf)
        if n > 1:
            put(a, 1, r, (j + 1) % n, 1, 17, -math.inf)
    seen = check(a)
    assert seen["inf"] >= GROUP and (max(lens) == 1 or seen["nan"])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_infinite_scores(lens, kind):
    """A score of +inf: its weight is inf / inf, so the outputs are NaN, and the sum of the exponentials is inf."""
    a = make(lens, kind)
    for r in range(0, len(lens), 2):
        a.q[r, 5 * DIM + 11] = math.inf
        if lens[r]:
            put(a, 0, r, lens[r] - 1, 1, 11, 0x38 if kind == "fp8" else 1.0)
    seen = check(a)
    rows = sum(1 for r in range(0, len(lens), 2) if lens[r])
    assert seen["lse_inf"] + seen["lse_nan"] == rows      # NaN where an FP8 key's code is 0
    assert kind == "fp8" or seen["lse_inf"] == rows


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [40, 1, 0, 5], [3000]])
def test_every_score_minus_infinity(lens, kind):
    a = make(lens, kind)
    for r, n in enumerate(lens):
        a.q[r, 2 * DIM + 1] = math.inf
        for j in range(n):
            put(a, 0, r, j, 0, 1, 0xB8 if kind == "fp8" else -1.0)
    seen = check(a)
    assert seen["none"] == sum(n > 0 for n in lens)


@pytest.mark.parametrize("lens", [[1], [40, 1, 0, 5], [3000]])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_no_weight_beside_values_that_are_not_finite(lens, value):
    """Zeros all the same: none of them has a weight in that head; in the others they count."""
    a = make(lens)
    for r, n in enumerate(lens):
        a.q[r, 2 * DIM + 1] = math.inf
        for j in range(n):
            put(a, 0, r, j, 0, 1, -1.0)
        if n:
            put(a, 1, r, n // 2, 0, 20, value)
    seen = check(a)
    rows = sum(n > 0 for n in lens)
    assert seen["none"] == rows and seen["nan"] == (rows * (GROUP - 1) if math.isnan(value) else 0)


@pytest.mark.parametrize("n", [40, 5000])
def test_infinite_value_of_a_small_weight(n):
    """Both parts of a weight are above zero down to 2^-110 of the largest, so its infinite v shows."""
    drops = [3.0, 30.7, 60.3, 90.1, 100.9, 105.6, 108.2, 109.0]
    a = make([n])
    a.q.zero_()
    for h, drop in enumerate(drops):
        a.q[0, h * DIM] = -drop * math.log(2.0) / a.scale      # BF16: within 2^-8 of it, above 2^-110
    for g in range(HEADS):
        for j in range(n):
            put(a, 0, 0, j, g, 0, 1.0 if j == n // 3 else 0.0)
        put(a, 1, 0, n // 3, g, 5, math.inf)
        put(a, 1, 0, n // 3, g, 6, -math.inf)
    seen = check(a)
    assert seen["inf"] == len(drops) and seen["nan"] == 0
