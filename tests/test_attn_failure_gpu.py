"""The failure path of the attention kernels, made to run on purpose without a fault: a test build (GEMV_DEBUG_DROP_X)
never issues the copies of V (in the kernels with tensor copies), or never counts a query's copies in (in the
others), so a warp's first wait for them runs out (2^14 rounds in that build). Every row gets NaN, whoever finishes it: a
warp, a CTA's join, the last CTA of a row, either level of a long row. The status bit is set, the workspace is left as a
call leaves it, and the regular library computes right after, in the same process."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding, build_lib
from tests import attn_util as au

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def drop_lib():
    return build_lib.build_debug_drop_x()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [16, 7])                       # tensor copies, copies by every thread
@pytest.mark.parametrize("lens", [[1], [20] * 300, [300, 0, 40, 5], [2000, 9], [40000]])
def test_wait_runs_out_and_reports(drop_lib, kind, page, lens):
    cache = au.Cache(lens, page, 2, 64, kind, seed=5)
    a = au.Attn(lens, cache, 8)
    with binding.use_library(drop_lib):
        a.run()                                                # returns GEMV_OK: the launch itself is fine
        torch.cuda.synchronize()
        assert binding.gemv_device_status() == binding.GEMV_STATUS_WAIT_TIMEOUT
        assert binding.gemv_device_status() == 0               # cleared by the read
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
