"""How many bits the attention's weights have when they meet V."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au

pytestmark = pytest.mark.gpu


def half_step(x):
    """Half the distance of BF16 numbers (8 bits) around x."""
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 9)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 12, 32])
@pytest.mark.parametrize("n", [40, 300, 3000])
def test_weights(kind, dim, group, n):
    """One token has score d_h, all others 0, and v = 0 at that token and positive at the others, so every output is
    one weight, exp(-d_h), times a sum: an error of that weight moves all columns alike.

    A single BF16 weight would be off by up to 2^-8, which with the rounding of the output is more than half a step.
    Allowed beside that half step: weights of 2^-16 (BF16 in two parts: the second takes up to 2^-7 of the weight and
    is rounded to 8 bits) or FP16's 2^-11; scores that are one product each, so three roundings of 2^-24 of d_h <= 10
    and in powers of two 2^-20; exp2's 2^-21; the FP32 sums of attn_bounds, numerator and denominator."""
    cache = au.Cache([n], 16, 1, dim, kind, seed=n)
    top = n // 3
    for which in range(2):
        view, val = cache.view(which), cache.values[which][0]
        for b in range(-(-n // 16)):
            rows = view[int(cache.table[0, b]), :min(16, n - 16 * b), 0]
            at = val[16 * b:16 * b + rows.shape[0], 0]
            if which == 0:
                rows.zero_()
                at.zero_()
            else:
                rows.copy_(rows & 0x7F if kind == "fp8" else rows.abs())
                at.abs_()
        if which == 0:
            view[int(cache.table[0, top // 16]), top % 16, 0, 0] = 0x38 if kind == "fp8" else 1.0
            val[top, 0, 0] = float(cache.scales[0][0].double()) if kind == "fp8" else 1.0
        else:
            view[int(cache.table[0, top // 16]), top % 16, 0] = 0
            val[top] = 0.0
    k0 = float(cache.values[0][0][top, 0, 0])
    q = torch.zeros(1, group, dim, dtype=torch.bfloat16)
    q[0, :, 0] = (torch.linspace(0.3, 9.9, group) / k0).bfloat16()
    a = au.Attn([n], cache, group, q=q.cuda(), scale=1.0)
    a.run()
    torch.cuda.synchronize()
    out, _, mass, _ = au.attend(q[0], cache.values[0][0], cache.values[1][0], 1.0)
    total = (n / 16 + 64) * 2.0 ** -23
    rel = (2.0 ** -16 if kind == "bf16" else au.FP16) + 2 * (2.0 ** -20 + 2.0 ** -21 + total)
    tol = half_step(out * (1 + rel)) + rel * mass
    err = (a.out[0].double().cpu().view(group, dim) - out).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert binding.gemv_device_status() == 0
