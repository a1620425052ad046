"""The rotary kernel that takes two tokens a block, at odd counts of tokens (its last block has one) and a pair of
columns at a time."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import test_rope_gpu as rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,q_heads,heads,dim,rot,axes,pad,offset", [
    (2501, 16, 2, 96, 96, 2, 0, 0), (1301, 8, 4, 80, 40, 1, 0, 0),     # BF16 rows turned by 40: a pair at a time
    (1300, 8, 4, 80, 40, 2, 4, 0), (901, 16, 8, 64, 64, 1, 0, 1), (4097, 2, 1, 254, 250, 1, 1, 0),
])
def test_two_tokens_a_block(f32, interleaved, T, q_heads, heads, dim, rot, axes, pad, offset):
    rope.test_rope(f32, interleaved, T, q_heads, heads, dim, rot, axes, pad, offset)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,q_heads,heads,dim,rot,page", [(701, 14, 2, 256, 256, 64), (1501, 8, 2, 80, 40, 24)])
def test_append_two_tokens_a_block(kind, layout, f32, T, q_heads, heads, dim, rot, page):
    """The last token, alone in its block, is padding."""
    rope.test_append(kind, layout, f32, T, q_heads, heads, dim, rot, page)


@pytest.mark.parametrize("rot", [128, 40])
def test_last_token_alone_in_place(rot):
    T = 1001
    c = rope.Case(T, 8, 2, 128, rot, f32=False, seed=4)
    want_q, size_q = c.turned(c.q, 8)
    want_k, size_k = c.turned(c.k, 2)
    binding.gemv_rope(c.args(q_out=c.q, k_out=c.k, k_out_stride=c.sk))
    torch.cuda.synchronize()
    rope.close(c.q.view(T, 8, 128), want_q, size_q)
    rope.close(c.k.view(T, 2, 128), want_k, size_k)
