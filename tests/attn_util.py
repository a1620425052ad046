"""Helpers for the tests of the decode step's attention half: paged caches,
references in 64 bits, and the error bounds the kernels are held to."""
from __future__ import annotations

import math

import torch

from memory_bound_decode_gb300 import binding

BF16 = 2.0 ** -8      # half a step, relative (torch.finfo(torch.bfloat16).eps / 2)
FP16 = 2.0 ** -11
E4M3 = 2.0 ** -4
F32 = 2.0 ** -24


def randn(seed: int, *shape, device="cuda", dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(device)


class Cache:
    """A pool with NaN in every slot that no request reaches, and its record."""

    def __init__(self, lens, page, heads, dim, kind="bf16", layout="token", seed=0, extra=0, width=None, spare=2,
                 device="cuda"):
        """``extra``: unused elements behind each page. Values as FP64 in ``values`` (k, v), token by token."""
        self.kind, self.page, self.heads, self.dim = kind, page, heads, dim
        R = len(lens)
        have = [-(-max(0, n) // page) for n in lens]
        self.num_pages = sum(have) + spare
        self.width = width or max(1, max(have))
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        order = torch.randperm(self.num_pages, generator=g).tolist()
        table = torch.full((R, self.width), -7, dtype=torch.int32)
        at = 0
        for r in range(R):
            table[r, :have[r]] = torch.tensor(order[at:at + have[r]], dtype=torch.int32)
            at += have[r]
        self.table = table.to(device)
        self.slot_stride, self.head_stride = (heads * dim, dim) if layout == "token" else (dim, page * dim)
        self.page_stride = page * heads * dim + extra
        self.scales = [None, None]
        self.pools, self.values = [], []
        for which in range(2):
            if kind == "fp8":
                pool = torch.full((self.num_pages * self.page_stride,), 0x7F, dtype=torch.uint8)
                self.scales[which] = torch.rand(heads, generator=g) * 0.05 + 0.01
            else:
                pool = torch.full((self.num_pages * self.page_stride,), float("nan"), dtype=torch.bfloat16)
            view = torch.as_strided(pool, (self.num_pages, page, heads, dim),
                                    (self.page_stride, self.slot_stride, self.head_stride, 1))
            vals = []
            for r in range(R):
                n = max(0, lens[r])
                x = torch.randn(n, heads, dim, generator=g)
                if kind == "fp8":
                    code = (x * 30).to(torch.float8_e4m3fn)
                    rows, val = code.view(torch.uint8), code.double() * self.scales[which].double()[:, None]
                else:
                    rows = x.to(torch.bfloat16)
                    val = rows.double()
                for b in range(have[r]):
                    part = rows[b * page:(b + 1) * page]
                    view[int(table[r, b]), :part.shape[0]] = part
                vals.append(val)
            self.pools.append(pool.to(device))
            self.values.append(vals)
        self.scales = [s.to(device) if s is not None else None for s in self.scales]

    def record(self, **over):
        f = dict(num_pages=self.num_pages, page_size=self.page, kv_heads=self.heads, head_dim=self.dim,
                 page_stride=self.page_stride, head_stride=self.head_stride, slot_stride=self.slot_stride,
                 kind=binding.GEMV_CACHE_FP8 if self.kind == "fp8" else binding.GEMV_CACHE_BF16,
                 k_scale=self.scales[0], v_scale=self.scales[1])
        f.update(over)
        return binding.kv_cache(self.pools[0], self.pools[1], **f)

    def view(self, which):
        return torch.as_strided(self.pools[which], (self.num_pages, self.page, self.heads, self.dim),
                                (self.page_stride, self.slot_stride, self.head_stride, 1))


def attend(q, k, v, scale, softcap=0.0):
    """One request in 64 bits: q [Hq, D], k and v [n, Hk, D] (visible tokens only). Returns out, lse, the weighted
    sum of |v| and the largest scale * sum |q k| of a head."""
    Hq, D = q.shape
    n, Hk, _ = k.shape
    G = Hq // Hk
    qg = q.double().view(Hk, G, D)
    s = torch.einsum("hgd,nhd->hgn", qg, k) * scale
    size = torch.einsum("hgd,nhd->hgn", qg.abs(), k.abs()).amax(-1) * abs(scale)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    out = torch.einsum("hgn,nhd->hgd", p, v)
    mass = torch.einsum("hgn,nhd->hgd", p, v.abs())
    return out.reshape(Hq, D), z.reshape(Hq), mass.reshape(Hq, D), size.reshape(Hq)


def attn_bounds(out, lse, mass, size, n, D, kind):
    """How far a kernel's output and lse may be from the 64-bit ones, element by element.

    A score is a sum of D products in FP32, each addition off by at most 2^-23 of the running sum (the matrix
    instructions may cut instead of round), bounded by the sum of the products' sizes, `size`; scaling and the
    change to powers of two add 2^-22 of the score. FP8: the parts of q below 2^-24 of its head's largest value are
    cut in FP16, at most D * 2^-24 times a code of at most 448 each, kept below the same 2^-23 by q's own size in
    these tests. Weights are off by that (absolutely, in
    the exponent) plus 2^-21 of exp2; they meet V with 2^-17 (two BF16 parts) or FP16's half step. Sums over n
    tokens add n / 16 + 64 roundings (16 tokens an instruction, then warps and pieces). Numerator and denominator
    each carry the weights' error. The output is then rounded to BF16."""
    score = (2 * D * 2.0 ** -23 + 2.0 ** -22) * size
    total = (n / 16 + 64) * 2.0 ** -23
    weight = 2.0 ** -17 if kind == "bf16" else FP16
    rel = 2 * (score + 2.0 ** -21 + total)[:, None] + weight
    return BF16 * out.abs() + (1 + BF16) * rel * mass + 1e-30, score + 2.0 ** -21 + total + 2.0 ** -22 * lse.abs()


class Attn:
    """One call of gemv_attn_decode with guarded outputs."""

    def __init__(self, lens, cache: Cache, q_heads, seed=1, scale=None, softcap=0.0, window=0, lse=True,
                 token_start=None, rows=None, pad=0, workspace=None, device="cuda", q=None, table=None, width=None):
        R, D = len(lens), cache.dim
        self.lens, self.cache, self.window, self.softcap, self.q_heads = lens, cache, window, softcap, q_heads
        self.scale = D ** -0.5 if scale is None else scale
        self.rows = rows if rows is not None else R
        self.stride = q_heads * D + pad
        full = randn(seed, max(1, self.rows), self.stride, device=device, dtype=torch.bfloat16, scale=2.0)
        if q is not None:
            full[:, :q_heads * D] = q.reshape(self.rows, -1)
        self.q = full
        self.guard = torch.full((self.rows + 2, self.stride), -777.0, dtype=torch.bfloat16, device=device)
        self.out = self.guard[1:-1]
        self.lse = torch.full((max(1, self.rows), q_heads), -777.0, device=device) if lse else None
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=device)
        self.token_start = (torch.tensor(token_start, dtype=torch.int32, device=device)
                            if token_start is not None else None)
        self.ws = workspace if workspace is not None else binding.attn_workspace(q_heads, cache.heads, D,
                                                                                 device=device)
        self.args = binding.attn_args(
            q=self.q, out=self.out, lse=self.lse, lens=self.lens_t, requests=R, q_heads=q_heads,
            q_stride=self.stride, out_stride=self.stride, table=cache.table if table is None else table,
            table_width=width or cache.width, table_stride=cache.width, scale=self.scale, softcap=softcap,
            window=window, workspace=self.ws, token_start=self.token_start, rows=self.rows)
        self.rec = cache.record()

    def run(self, stream=None):
        binding.gemv_attn_decode(self.args, self.rec, stream)

    def check(self, written=None, lens=None):
        """Every written row against the 64-bit reference, every other byte as it was."""
        lens = self.lens if lens is None else lens
        Hq, D = self.q_heads, self.cache.dim
        got = self.guard.double().cpu()
        lse = self.lse.double().cpu() if self.lse is not None else None
        mark = float(torch.tensor(-777.0).bfloat16())
        assert (got[0] == mark).all() and (got[-1] == mark).all(), "write outside out"
        assert (got[1:-1, Hq * D:] == mark).all(), "write between rows"
        row_of = {}
        for r in range(len(lens)):
            if self.token_start is not None:
                a, b = int(self.token_start[r]), int(self.token_start[r + 1])
                if b <= a:
                    continue
                row_of[b - 1] = r
            else:
                row_of[r] = r
        for row in range(self.rows):
            r = row_of.get(row)
            y = got[1 + row, :Hq * D].view(Hq, D)
            if r is None or lens[r] < 0:
                assert (y == mark).all(), f"row {row} was written"
                assert lse is None or (lse[row] == -777.0).all()
                continue
            n = lens[r]
            if n == 0:
                assert (y == 0).all() and (lse is None or (lse[row] == -math.inf).all())
                continue
            begin = max(0, n - self.window) if self.window else 0
            k, v = (self.cache.values[i][r][begin:n] for i in range(2))
            q = self.q[row, :Hq * D].cpu().view(Hq, D)
            out, z, mass, size = attend(q, k, v, self.scale, self.softcap)
            tol, tol_z = attn_bounds(out, z, mass, size, n - begin, D, self.cache.kind)
            err = (y - out).abs()
            assert (err <= tol).all(), (row, n, float((err / tol).max()), float(err.max()))
            if lse is not None:
                ez = (lse[row] - z).abs()
                assert (ez <= tol_z).all(), (row, n, float((ez / tol_z).max()))


def turn(x, positions, inv, axis, rot, interleaved):
    """x [T, H, D] turned in 64 bits; positions [A, T]."""
    x = x.double().cpu().clone()
    pos = positions.double().cpu()
    half = rot // 2
    ang = pos[axis.long()].T * inv.double()[None, :]
    c, s = ang.cos()[:, None, :], ang.sin()[:, None, :]
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, w = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    size = torch.zeros_like(x)
    size[..., a] = size[..., b] = u.abs() + w.abs()
    return x, size
