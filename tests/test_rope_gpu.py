"""gemv_rope and gemv_rope_append against rotations in 64 bits."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests import attn_util as au

pytestmark = pytest.mark.gpu

# Sine, cosine and the rotation in FP32: the reduced angle is off by at most 2^-24 of half a turn, sinpi / cospi by a
# few units in the last place, the products and the sum by a rounding each: below 2^-20 of |a| + |b|.
TURN = 2.0 ** -20


class Case:
    def __init__(self, T, q_heads, heads, dim, rot, axes=1, interleaved=False, f32=True, far=5000, seed=0, pad=0,
                 offset=0):
        dt = torch.float32 if f32 else torch.bfloat16
        self.T, self.q_heads, self.heads, self.dim, self.rot = T, q_heads, heads, dim, rot
        self.interleaved, self.f32, self.axes = interleaved, f32, axes
        self.sq, self.sk = q_heads * dim + pad, heads * dim + pad

        def rows(i, stride):
            x = au.randn(seed * 10 + i, T * stride + offset, dtype=dt)
            return x[offset:].view(T, stride)
        self.q, self.k, self.v = rows(1, self.sq), rows(2, self.sk), rows(3, self.sk)
        half = rot // 2
        self.inv = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(half)], dtype=torch.float64)
        g = torch.Generator().manual_seed(seed)
        self.axis = torch.randint(0, axes, (half,), generator=g, dtype=torch.int32)
        self.pos = torch.randint(-3 if far > 10 else 0, far, (axes, T), generator=g, dtype=torch.int32).cuda()
        self.freqs = binding.rope_freqs(self.inv, device="cuda")
        self.q_out = torch.full((T, self.sq), -777.0, dtype=torch.bfloat16, device="cuda")
        self.k_out = torch.full((T, self.sk), -777.0, dtype=torch.bfloat16, device="cuda")

    def args(self, **over):
        f = dict(q=self.q, k=self.k, q_out=self.q_out, positions=self.pos, freqs=self.freqs, tokens=self.T,
                 q_heads=self.q_heads, kv_heads=self.heads, head_dim=self.dim, rot_dim=self.rot, q_stride=self.sq,
                 k_stride=self.sk, q_out_stride=self.sq, rows=binding.GEMV_ROWS_F32 if self.f32
                 else binding.GEMV_ROWS_BF16, pairs=binding.GEMV_PAIRS_INTERLEAVED if self.interleaved
                 else binding.GEMV_PAIRS_HALF, axes=self.axes, axis_stride=self.T,
                 pair_axis=self.axis.cuda() if self.axes > 1 else None)
        f.update(over)
        return binding.rope_args(**f)

    def turned(self, rows, heads):
        x = rows[:, :heads * self.dim].reshape(self.T, heads, self.dim)
        return au.turn(x, self.pos, self.inv, self.axis if self.axes > 1 else torch.zeros_like(self.axis), self.rot,
                       self.interleaved)


def close(got, want, size):
    tol = au.BF16 * want.abs() + (1 + au.BF16) * TURN * size + 1e-38
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,q_heads,heads,dim,rot,axes,pad,offset", [
    (1, 1, 1, 128, 128, 1, 0, 0), (3, 32, 8, 128, 128, 1, 0, 0), (5, 7, 7, 80, 80, 2, 0, 0),
    (17, 4, 2, 256, 64, 3, 8, 0), (9, 5, 1, 64, 32, 1, 4, 0), (4, 3, 1, 72, 18, 2, 2, 0), (2, 2, 2, 2, 2, 1, 0, 0),
    (6, 4, 2, 64, 64, 8, 0, 1), (2500, 16, 2, 96, 96, 2, 0, 0), (3, 2, 1, 254, 250, 1, 1, 0),
])
def test_rope(f32, interleaved, T, q_heads, heads, dim, rot, axes, pad, offset):
    c = Case(T, q_heads, heads, dim, rot, axes, interleaved, f32, seed=T + dim, pad=pad, offset=offset)
    binding.gemv_rope(c.args(k_out=c.k_out, k_out_stride=c.sk))
    torch.cuda.synchronize()
    mark = float(torch.tensor(-777.0).bfloat16())
    for rows, out, n in ((c.q, c.q_out, q_heads), (c.k, c.k_out, heads)):
        want, size = c.turned(rows, n)
        close(out[:, :n * dim].view(T, n, dim), want, size)
        assert (out[:, n * dim:].float() == mark).all()


def test_rope_in_place():
    c = Case(33, 8, 2, 128, 128, f32=False, seed=4)
    want_q, size_q = c.turned(c.q, 8)
    want_k, size_k = c.turned(c.k, 2)
    binding.gemv_rope(c.args(q_out=c.q, k_out=c.k, k_out_stride=c.sk))
    torch.cuda.synchronize()
    close(c.q.view(33, 8, 128), want_q, size_q)
    close(c.k.view(33, 2, 128), want_k, size_k)


def test_far_positions():
    """The angle is reduced exactly: position 2^31 - 1 is as accurate as position 1."""
    c = Case(4, 2, 1, 64, 64, seed=6)
    c.pos.copy_(torch.tensor([[1, 1 << 20, 2 ** 31 - 1, -(2 ** 31)]], dtype=torch.int32))
    binding.gemv_rope(c.args(k_out=c.k_out, k_out_stride=c.sk))
    torch.cuda.synchronize()
    # 64 bits themselves are off by 2^31 * 2^-53 * a few in the angle at the far end: 2^-20 of |a| + |b|, as TURN is.
    want, size = c.turned(c.q, 2)
    close(c.q_out.view(4, 2, 64), want, 2 * size)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,q_heads,heads,dim,rot,page", [
    (1, 32, 8, 128, 128, 16), (37, 8, 2, 80, 48, 24), (5, 4, 4, 64, 64, 1), (700, 14, 2, 256, 256, 64),
    (9, 3, 1, 96, 6, 7),
])
def test_append(kind, layout, f32, T, q_heads, heads, dim, rot, page):
    """Every slot written as it should be, every other byte of the pool and the rows of padding tokens as they were."""
    c = Case(T, q_heads, heads, dim, rot, f32=f32, seed=T)
    cache = au.Cache([T + 3 * page], page, heads, dim, kind, layout, seed=7, extra=16)
    g = torch.Generator().manual_seed(3)
    total = cache.num_pages * page
    slots = torch.randperm(total, generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[1], slots[T - 1] = -1, total              # padding: negative, and past the pool
    before = [p.clone() for p in cache.pools]
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=slots.cuda()), cache.record())
    torch.cuda.synchronize()
    mark = float(torch.tensor(-777.0).bfloat16())
    live = (slots >= 0) & (slots < total)
    want, size = c.turned(c.q, q_heads)
    got = c.q_out.view(T, q_heads, dim)
    close(got[live.cuda()], want[live], size[live])
    assert (got[(~live).cuda()].float() == mark).all()
    at = slots[live].long()
    for which, rows in ((0, c.k), (1, c.v)):
        if which == 0:
            want, size = c.turned(rows, heads)
        else:
            want = rows[:, :heads * dim].reshape(T, heads, dim).double().cpu()
            size = torch.zeros_like(want)
        want, size = want[live], size[live]
        view = cache.view(which)
        got = view[(at // page).cuda(), (at % page).cuda()].cpu()
        if kind == "bf16":
            close(got, want, size)
        else:
            sc = cache.scales[which].double().cpu()[:, None]
            w = (want / sc).clamp(-448, 448)
            # half a step of E4M3: 2^-4 of the value, at least half its smallest step (2^-10); and the FP32 errors
            tol = (au.E4M3 * w.abs()).clamp(min=2.0 ** -10) + 1.07 * (TURN * size + 2 * au.F32 * want.abs()) / sc
            err = (got.view(torch.float8_e4m3fn).double() - w).abs()
            assert (err <= tol).all(), float((err / tol).max())
        # untouched: put the old rows back, then the pools are the same bytes
        pages, offs = (at // page).cuda(), (at % page).cuda()
        old = torch.as_strided(before[which], view.shape, view.stride())
        bits = torch.uint8 if kind == "fp8" else torch.int16
        view.view(bits)[pages, offs] = old.view(bits)[pages, offs]
        assert torch.equal(cache.pools[which].view(bits), before[which].view(bits))


def test_append_fp8_saturates_and_keeps_nan():
    c = Case(2, 1, 1, 64, 64, f32=True, seed=1)
    c.pos.zero_()
    cache = au.Cache([16], 16, 1, 64, "fp8")
    c.v[0, :4] = torch.tensor([1e30, -float("inf"), float("nan"), 0.0])
    binding.gemv_rope_append(c.args(v=c.v, v_stride=c.sk, slots=torch.tensor([5, 9], dtype=torch.int32).cuda()),
                             cache.record())
    torch.cuda.synchronize()
    got = cache.view(1)[0, 5, 0, :4].view(torch.float8_e4m3fn).float().cpu()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 0


def test_captured():
    c = Case(8, 4, 2, 64, 64, seed=2)
    args = c.args(k_out=c.k_out, k_out_stride=c.sk)
    binding.gemv_rope(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gemv_rope(args)
    c.pos.add_(11)
    graph.replay()
    torch.cuda.synchronize()
    want, size = c.turned(c.q, 4)
    close(c.q_out.view(8, 4, 64), want, size)


def test_no_tokens():
    c = Case(3, 4, 2, 64, 64, seed=2)
    binding.gemv_rope(c.args(k_out=c.k_out, k_out_stride=c.sk, tokens=0))
    torch.cuda.synchronize()
    assert (c.q_out.float() == float(torch.tensor(-777.0).bfloat16())).all()
