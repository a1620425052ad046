"""Requests that gemv_block_tables refuses, through the rest of a step: attention gives them zeros instead of what an
earlier step left in their rows."""
import math

import pytest
import torch

from memory_bound_decode_gb300 import binding, workloads
from tests import attn_util as au

pytestmark = pytest.mark.gpu

TINY = dict(layers=2, hidden=512, intermediate=512, vocab=64, q_rows=512, kv_rows=256)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("requests", [5, 40, 300])
def test_refused_requests_get_zeros(requests, starts, kind):
    lens = [(i * 53) % 400 for i in range(requests)]
    lens[2] = 1500
    cache = au.Cache(lens, 16, 2, 64, kind, seed=3)
    status = [(0, 1, 0, 2, 4, 0, 3)[i % 7] for i in range(requests)]
    kw = {}
    if starts:
        first = [0]
        for i in range(requests):
            first.append(first[-1] + (0 if i % 11 == 5 else 1 + i % 2))
        kw = dict(token_start=first, rows=first[-1])
    a = au.Attn(lens, cache, 8, **kw)
    keep = i32(status)
    a.args.status = keep.data_ptr()
    a.run()
    torch.cuda.synchronize()
    a.check(lens=[0 if s else n for s, n in zip(status, lens)])
    assert binding.gemv_device_status() == 0


def test_row_of_a_refused_request_past_the_outputs_is_no_bad_page():
    """Status 3: its tokens end past max_tokens, so its row lies past q and out."""
    lens = [30, 40]
    cache = au.Cache(lens, 16, 2, 64, seed=3)
    a = au.Attn(lens, cache, 8, token_start=[0, 1, 9], rows=2)
    keep = i32([0, 3])
    a.args.status = keep.data_ptr()
    binding.gemv_device_status()
    a.run()
    torch.cuda.synchronize()
    assert binding.gemv_device_status() == 0
    mark = float(torch.tensor(-777.0).bfloat16())
    assert (a.out[1].float() == mark).all() and (a.out[0].float() != mark).all()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True])
def test_refused_request_of_a_step(cache, captured):
    """From the first step on, and after steps that were served: zeros in, zeros through the output projection."""
    lens = [32, 31, 5]                             # rows of two pages: the first is full, the second has one place
    step = workloads.AttentionStep(TINY, lens, batch=3, cache=cache, page_size=16, advance=True, room=0)
    for d in step.layers:
        d["q"].fill_(3.0)
        d["out"].fill_(math.nan)
        d["o"].fill_(math.nan)
    if captured:
        first = workloads.AttentionStep(TINY, [1], batch=1, cache=cache)
        first.run()                                # the library is set up
        torch.cuda.synchronize()
        step.capture()
    for served in ([False, True, True], [False, False, True]):
        if captured:
            step.launch()
        else:
            step.run()
        torch.cuda.synchronize()
        assert step.status.tolist() == [0 if s else 2 for s in served]
        for d in step.layers:
            for r, s in enumerate(served):
                assert torch.isfinite(d["out"][r].float()).all() and torch.isfinite(d["o"][r]).all()
                assert bool((d["out"][r] != 0).any()) == s and bool((d["o"][r] != 0).any()) == s
    assert binding.gemv_device_status() == 0
