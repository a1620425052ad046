"""An FP8 cache with a scale for each block of tokens and head, for tests: pools
with NaN codes and NaN scales wherever no request reaches, and the write's
definition token by token."""
from __future__ import annotations

import math

import torch

from memory_bound_decode_gb300 import binding

FLOOR = 2.0 ** -30
MAX = 448.0


def code_of(x):
    """The nearest E4M3 codes of values (any float tensor on the CPU), at most 448 in magnitude, NaN as it is."""
    return x.float().clamp(-MAX, MAX).to(torch.float8_e4m3fn)


def need(a: float) -> float:
    """The smallest power of two that is at least a / 448, no smaller than the floor."""
    if a <= 0:
        return FLOOR
    m, e = math.frexp(a)                      # a = m 2^e, 448 = 0.875 * 2^9
    return max(FLOOR, math.ldexp(1.0, e - 9 if m <= 0.875 else e - 8))


class BlockCache:
    kind = "fp8"                              # of the error bounds

    def __init__(self, lens, page, block, heads, dim, layout="token", seed=0, extra=0, width=None, spare=2,
                 spread=(-9, -3), powers=True, device="cuda", fill=True):
        """``extra``: unused elements behind each page (and scales behind each page's). Scales 2^e with e from
        ``spread``, or (``powers`` false) anything between. ``fill``: the requests' tokens hold values."""
        self.page, self.block, self.heads, self.dim, self.device = page, block, heads, dim, device
        R = len(lens)
        have = [-(-max(0, n) // page) for n in lens]
        self.num_pages = sum(have) + spare
        self.width = width or max(1, max(have))
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.host_table = torch.full((R, self.width), -7, dtype=torch.int32)
        at = 0
        for r in range(R):
            self.host_table[r, :have[r]] = torch.tensor(order[at:at + have[r]], dtype=torch.int32)
            at += have[r]
        self.table = self.host_table.to(device)
        per = page // block
        token = layout == "token"
        self.slot_stride, self.head_stride = (heads * dim, dim) if token else (dim, page * dim)
        self.page_stride = page * heads * dim + extra
        self.scale_block_stride, self.scale_head_stride = (heads, 1) if token else (1, per)
        self.scale_page_stride = per * heads + extra
        self.pools, self.scales, self.values = [], [], []
        for _ in range(2):
            pool = torch.full((self.num_pages * self.page_stride,), 0x7F, dtype=torch.uint8)
            scale = torch.full((self.num_pages * self.scale_page_stride,), math.nan)
            codes, scales = self.codes_of(pool), self.scales_of(scale)
            vals = []
            for r in range(R):
                n = max(0, lens[r]) if fill else 0
                x = code_of(torch.randn(n, heads, dim, generator=g) * 40)
                v = torch.zeros(n, heads, dim, dtype=torch.float64)
                for b in range(-(-n // block)):
                    j = slice(b * block, min(n, (b + 1) * block))
                    pg, place = int(self.host_table[r, b * block // page]), b * block % page
                    e = torch.rand(heads, generator=g) * (spread[1] - spread[0]) + spread[0]
                    s = torch.exp2(e.round()) if powers else torch.exp2(e)
                    scales[pg, place // block] = s
                    codes[pg, place:place + j.stop - j.start] = x[j].view(torch.uint8)
                    v[j] = x[j].double() * s.double()[None, :, None]
                vals.append(v)
            self.pools.append(pool.to(device))
            self.scales.append(scale.to(device))
            self.values.append(vals)

    def codes_of(self, pool):
        """[page, slot, head, column]"""
        return torch.as_strided(pool, (self.num_pages, self.page, self.heads, self.dim),
                                (self.page_stride, self.slot_stride, self.head_stride, 1))

    def scales_of(self, scale):
        """[page, block, head]"""
        return torch.as_strided(scale, (self.num_pages, self.page // self.block, self.heads),
                                (self.scale_page_stride, self.scale_block_stride, self.scale_head_stride))

    def record(self, **over):
        f = dict(num_pages=self.num_pages, page_size=self.page, kv_heads=self.heads, head_dim=self.dim,
                 page_stride=self.page_stride, head_stride=self.head_stride, slot_stride=self.slot_stride,
                 kind=binding.GEMV_CACHE_FP8_BLOCK, block_tokens=self.block, k_block_scale=self.scales[0],
                 v_block_scale=self.scales[1], scale_page_stride=self.scale_page_stride,
                 scale_block_stride=self.scale_block_stride, scale_head_stride=self.scale_head_stride)
        f.update(over)
        return binding.kv_cache(self.pools[0], self.pools[1], **f)

    def slots_of(self, r, first, n):
        t = self.host_table
        return [int(t[r, j // self.page]) * self.page + j % self.page for j in range(first, first + n)]

    def host(self):
        """(codes, scales) of k and of v on the CPU, whole buffers."""
        return [(p.cpu().clone(), s.cpu().clone()) for p, s in zip(self.pools, self.scales)]


def write(cache: BlockCache, codes, scales, rows, slots, peak=None):
    """The write into the host buffers `codes` and `scales`: rows [T, H, D] (FP32, already turned) at their slots.
    `peak`: the largest magnitudes to go by, [T, H] (default: the rows' own)."""
    c, s = cache.codes_of(codes), cache.scales_of(scales)
    total, B = cache.num_pages * cache.page, cache.block
    finite = torch.where(torch.isfinite(rows), rows.abs(), torch.zeros_like(rows))
    peak = finite.amax(-1) if peak is None else peak
    t = 0
    while t < len(slots):
        slot = slots[t]
        if not 0 <= slot < total:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slot + n and (slot + n) % B != 0:
            n += 1
        page, place = slot // cache.page, slot % cache.page
        blk, held = place // B, place % B
        for h in range(cache.heads):
            new = need(float(peak[t:t + n, h].max()))
            old = float(s[page, blk, h])
            if held:
                m, e = math.frexp(old)
                new = max(old if m == 0.5 else math.ldexp(1.0, e), new)   # a power of two in any case
                if new > old:
                    at = c[page, place - held:place, h]
                    at.copy_(code_of(at.clone().contiguous().view(torch.float8_e4m3fn).float() * (old / new)).view(torch.uint8))
            s[page, blk, h] = new
            c[page, place:place + n, h] = code_of(rows[t:t + n, h] / new).view(torch.uint8)
        t += n
