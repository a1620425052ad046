"""A paged key-value cache in 8 bits whose scales are found as it is written, as
cases: the write (rotary positions, a scale for each block of tokens and head,
E4M3 codes), the read back into rows, and attention of one new token over it.
Each case runs either in its plain form (elementary torch operations in 32
bits, or in 64 where 32 lose what matters) or, with ``own`` true, through the
entry points of the package's binding.

Head counts, head size and page tables follow the decode step of this package
(32 query heads, 8 key-value heads, 128 columns a head); the others are generic.

A block is `block` neighbouring slots of a page. Its value is code times scale,
one scale per block and key-value head, K and V apart. New tokens of a block:
the scale becomes the smallest power of two that takes their largest value into
E4M3's range (448), but no smaller than it was if the block holds earlier
tokens, whose codes move with it.
"""
import math

import torch

own = False

DEV = "cuda"
SMALLEST = 2.0 ** -30          # of a block's scale


# ---- cases -----------------------------------------------------------------

def listed():
    heads = dict(q_heads=32, kv_heads=8, dim=128)
    return [
        # The new token of 16 requests: most fall into a block that earlier tokens have begun, some make its scale grow.
        dict(name="append-decode", op="append", requests=16, lo=100, hi=4100, new_lo=1, new_hi=1, pad=0, **heads,
             rot=128, axes=1, pairs="half", rows="f32", layout="token", page=16, block=16),
        # A large batch with larger blocks, rows already in BF16, two of them padding.
        dict(name="append-decode-256", op="append", requests=254, lo=1, hi=1000, new_lo=1, new_hi=1, pad=2, **heads,
             rot=128, axes=1, pairs="half", rows="bf16", layout="head", page=64, block=32),
        # Prompts of all lengths, some of them going on in a block that is begun, with a ragged end of padding rows.
        dict(name="append-prompts", op="append", requests=9, lo=0, hi=500, new_lo=1, new_hi=900, pad=33, **heads,
             rot=128, axes=1, pairs="half", rows="f32", layout="token", page=32, block=16),
        # An image between text, three axes of positions, one long piece, blocks of a whole page.
        dict(name="append-axes", op="append", requests=1, lo=37, hi=37, new_lo=1021, new_hi=1021, pad=5, **heads,
             rot=128, axes=3, pairs="half", rows="bf16", layout="head", page=64, block=64),
        # The prefix of one short request, for the next piece of its prompt.
        dict(name="read-1x300", op="read", requests=1, lo=300, hi=300, part=1.0, kv_heads=8, dim=128, out="bf16",
             kind="block", layout="token", page=16, block=16, pad=0),
        # Prefixes of a batch, a request without any among them.
        dict(name="read-16x4k", op="read", requests=16, lo=0, hi=4096, part=1.0, kv_heads=8, dim=128, out="bf16",
             kind="block", layout="token", page=16, block=16, pad=7),
        # The second half of every context as FP32 rows, heads of 80 columns, pages that are no power of two.
        dict(name="read-32x16k-f32", op="read", requests=32, lo=1, hi=16384, part=0.5, kv_heads=8, dim=80, out="f32",
             kind="block", layout="head", page=24, block=8, pad=0),
        # The latency of one request with a short context.
        dict(name="attn-1x1000", op="attn", requests=1, lo=1000, hi=1000, **heads, layout="token", page=16, block=16,
             window=0, softcap=0.0, lse=True),
        # An ordinary batch with contexts of all lengths, a request without any among them.
        dict(name="attn-16x4k", op="attn", requests=16, lo=0, hi=4096, **heads, layout="token", page=16, block=16,
             window=0, softcap=0.0, lse=False),
        # A large batch with long contexts.
        dict(name="attn-64x32k", op="attn", requests=64, lo=16384, hi=32768, **heads, layout="head", page=64, block=32,
             window=0, softcap=0.0, lse=False),
        # One request with a very long context: nothing but the split over its length fills the GPU.
        dict(name="attn-1x131072", op="attn", requests=1, lo=131071, hi=131071, **heads, layout="head", page=64,
             block=64, window=0, softcap=0.0, lse=True),
        # Wide heads in groups of 16, a sliding window and capped scores, pages that divide no tile.
        dict(name="attn-wide-window", op="attn", requests=48, lo=0, hi=9000, q_heads=32, kv_heads=2, dim=256,
             layout="head", page=24, block=8, window=4096, softcap=50.0, lse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "append", "read", "read", "attn", "attn", "attn"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    block = rng.choice([b for b in (1, 8, 16, 16, 24, 32, 64) if page % b == 0])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 8, 16])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    case = dict(op=op, kv_heads=kv_heads, dim=dim, layout=rng.choice(["token", "head"]), page=page, block=block)
    if op == "append":
        q_heads = kv_heads * rng.choice([1, 2, 4, 4, 7, 8])
        most = max(64, min(8192, 4096 * 48 * 128 // ((q_heads + 2 * kv_heads) * dim)))
        requests = _log_int(rng, 1, 512)
        new_hi = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        while requests * new_hi > 2 * most:
            requests, new_hi = max(1, requests * 3 // 4), max(1, new_hi * 3 // 4)
        hi = _log_int(rng, 1, 1000)
        case.update(requests=requests, lo=rng.choice([0, 1, hi]), hi=hi, new_lo=rng.choice([1, new_hi]), new_hi=new_hi,
                    pad=rng.choice([0, 0, 1, 19]), q_heads=q_heads, rot=rng.choice([dim, dim, dim // 2]),
                    axes=rng.choice([1, 1, 2, 3]), pairs=rng.choice(["half", "half", "interleaved"]),
                    rows=rng.choice(["f32", "bf16"]))
        return case
    requests, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
    if op == "read":
        while requests * hi * kv_heads * dim > 16 * 16384 * 8 * 128:
            requests, hi = max(1, requests * 3 // 4), max(1, hi * 3 // 4)
        case.update(requests=requests, lo=rng.choice([0, 1, hi]), hi=hi, part=rng.choice([1.0, 1.0, 0.5, 0.1]),
                    out=rng.choice(["bf16", "bf16", "f32"]), kind=rng.choice(["block", "block", "block", "fp8", "bf16"]),
                    pad=rng.choice([0, 0, 5]))
        return case
    while requests * hi * kv_heads * dim > 64 * 24000 * 8 * 128:
        requests, hi = max(1, requests * 3 // 4), max(1, hi * 3 // 4)
    case.update(requests=requests, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi,
                q_heads=kv_heads * rng.choice([1, 2, 4, 4, 5, 8, 16, 32]),
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]), softcap=rng.choice([0.0, 0.0, 30.0]),
                lse=rng.choice([True, False]))
    return case


# ---- inputs ----------------------------------------------------------------

def _at(lo, hi, i, n):
    return hi if n == 1 else lo + (hi - lo) * i // (n - 1)


def _spaced(lo, hi, n, g):
    """n whole numbers from lo to hi, evenly spaced, in an order of the seed's: the same sum for every seed."""
    v = torch.tensor([_at(lo, hi, i, n) for i in range(n)], dtype=torch.int64)
    return v[torch.randperm(n, generator=g)]


def _gens(seed):
    g, gc = torch.Generator(device=DEV), torch.Generator(device="cpu")
    g.manual_seed(seed)
    gc.manual_seed(seed)
    return g, gc


def _pages(lens, P, width, g):
    """Page numbers of every request, in a shuffled order, and how many pages the pool has."""
    have = (lens + P - 1) // P
    held = int(have.sum())
    num_pages = int(lens.sum()) // P + lens.numel() + 3         # the same for every seed, and at least `held`
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < have[:, None]] = torch.randperm(num_pages, generator=g).to(torch.int32)[:held]
    return table, num_pages


def _pools(case, num_pages, g, kind="block"):
    """K and V pools with what earlier tokens left there: codes of values about 32 in size, and the scales."""
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    token = case["layout"] == "token"
    st = {}
    for n in ("k", "v"):
        x = torch.randn((num_pages, P, H, D) if token else (num_pages, H, P, D), generator=g, device=DEV, dtype=torch.bfloat16)
        st[n + "c"] = x if kind == "bf16" else (x * 32).to(torch.float8_e4m3fn)
        if kind == "block":
            B = P // case["block"]
            e = torch.randint(-8, -4, (num_pages, B, H) if token else (num_pages, H, B), generator=g, device=DEV)
            st[n + "s"] = torch.ldexp(torch.ones(e.shape, device=DEV), e)
        elif kind == "fp8":
            st[n + "s"] = (torch.rand(H, generator=g, device=DEV) + 0.5) / 32
    return st


def prepare(case, seed):
    return {"append": _prepare_append, "read": _prepare_read, "attn": _prepare_attn}[case["op"]](case, seed)


def _inv_freq(case):
    """base^(-2i / rot) for pair i, and the axis of pair i: equal shares of the pairs, the first axis's first."""
    half = case["rot"] // 2
    inv = torch.tensor([500000.0 ** (-2.0 * i / case["rot"]) for i in range(half)], dtype=torch.float64)
    axis = torch.tensor([min(i * case["axes"] // half, case["axes"] - 1) for i in range(half)], dtype=torch.int32)
    return inv, axis


def _prepare_append(case, seed):
    g, gc = _gens(seed)
    R, P, Hq, Hk, D = case["requests"], case["page"], case["q_heads"], case["kv_heads"], case["dim"]
    lens, new = _spaced(case["lo"], case["hi"], R, gc), _spaced(case["new_lo"], case["new_hi"], R, gc)
    width = -(-(case["hi"] + case["new_hi"]) // P)
    table, num_pages = _pages(lens + new, P, width, gc)
    live = int(new.sum())
    T = live + case["pad"]
    r = torch.repeat_interleave(torch.arange(R), new)
    pos = lens[r] + torch.arange(live) - (torch.cumsum(new, 0) - new)[r]
    slots = torch.full((T,), -1, dtype=torch.int32)
    slots[:live] = table[r, pos // P] * P + (pos % P).to(torch.int32)
    positions = torch.randint(0, 128, (case["axes"], T), generator=gc, dtype=torch.int32)
    positions[0, :live] = pos.to(torch.int32)
    # The blocks that get tokens, each token's, and the place of the first new token of each.
    blocks, of = torch.unique(slots[:live].long() // case["block"], return_inverse=True)
    first = torch.full((blocks.numel(),), case["block"]).scatter_reduce(0, of, slots[:live].long() % case["block"], "amin")
    dt = torch.float32 if case["rows"] == "f32" else torch.bfloat16
    row = lambda h, d=dt: torch.randn((T, h, D), generator=g, device=DEV, dtype=d)  # noqa: E731
    inv, axis = _inv_freq(case)
    st = dict(case=case, q=row(Hq), k=row(Hk), v=row(Hk), q_out=row(Hq, torch.bfloat16), slots=slots.to(DEV), live=live,
              positions=positions.to(DEV), inv=inv.to(DEV), axis=axis.to(DEV), blocks=blocks.to(DEV), of=of.to(DEV),
              first=first.to(DEV), num_pages=num_pages, **_pools(case, num_pages, g))
    st["outs"] = dict(q=st["q_out"], k=st["kc"], v=st["vc"], ks=st["ks"], vs=st["vs"])
    return st


def _prepare_read(case, seed):
    g, gc = _gens(seed)
    R, P, H, D = case["requests"], case["page"], case["kv_heads"], case["dim"]
    lens = _spaced(case["lo"], case["hi"], R, gc)
    table, num_pages = _pages(lens, P, max(1, -(-case["hi"] // P)), gc)
    count = torch.tensor([int(n * case["part"]) for n in lens.tolist()])     # the last tokens of each request
    row_start = torch.zeros(R + 1, dtype=torch.int32)
    row_start[1:] = torch.cumsum(count, 0)
    rows = int(row_start[-1]) + case["pad"]
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    st = dict(case=case, table=table.to(DEV), begin=(lens - count).to(DEV, torch.int32), row_start=row_start.to(DEV),
              rows=rows, num_pages=num_pages, **_pools(case, num_pages, g, case["kind"]))
    st["outs"] = {n: torch.randn((max(1, rows), H, D), generator=g, device=DEV, dtype=dt) for n in ("k", "v")}
    return st


def _prepare_attn(case, seed):
    g, gc = _gens(seed)
    R, Hq, D, P = case["requests"], case["q_heads"], case["dim"], case["page"]
    lens = _spaced(case["lo"], case["hi"], R, gc)
    table, num_pages = _pages(lens, P, max(1, -(-case["hi"] // P)), gc)
    st = dict(case=case, lens=lens.to(DEV, torch.int32), table=table.to(DEV), num_pages=num_pages,
              q=2 * torch.randn((R, Hq, D), generator=g, device=DEV, dtype=torch.bfloat16),
              **_pools(case, num_pages, g))
    st["outs"] = dict(out=torch.empty((R, Hq, D), device=DEV, dtype=torch.bfloat16))
    if case["lse"]:
        st["outs"]["lse"] = torch.empty((R, Hq), device=DEV, dtype=torch.float32)
    return st


# ---- one pass --------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn}[state["case"]["op"]](state)


def _own(st):
    """The package's calls. The argument records name buffers, as a serving loop's do, and are filled once."""
    if "call" not in st:
        st["call"] = _record(st)
    call, args, cache = st["call"]
    call(args, cache)
    return st["outs"]


def _record(st):
    from memory_bound_decode_gb300 import binding
    case, op = st["case"], st["case"]["op"]
    P, H, D, kind = case["page"], case["kv_heads"], case["dim"], case.get("kind", "block")
    token = case["layout"] == "token"
    more = {}
    if kind == "block":
        B = P // case["block"]
        more = dict(block_tokens=case["block"], k_block_scale=st["ks"], v_block_scale=st["vs"], scale_page_stride=B * H,
                    scale_block_stride=H if token else 1, scale_head_stride=1 if token else B)
    elif kind == "fp8":
        more = dict(k_scale=st["ks"], v_scale=st["vs"])
    cache = binding.kv_cache(
        st["kc"], st["vc"], num_pages=st["num_pages"], page_size=P, kv_heads=H, head_dim=D, page_stride=P * H * D,
        head_stride=D if token else P * D, slot_stride=H * D if token else D,
        kind={"bf16": binding.GEMV_CACHE_BF16, "fp8": binding.GEMV_CACHE_FP8, "block": binding.GEMV_CACHE_FP8_BLOCK}[kind],
        **more)
    if op == "append":
        Hq, T = case["q_heads"], st["slots"].numel()
        return binding.gemv_rope_append, binding.rope_args(
            q=st["q"], k=st["k"], v=st["v"], tokens=T, q_heads=Hq, kv_heads=H, head_dim=D, rot_dim=case["rot"],
            q_stride=Hq * D, k_stride=H * D, v_stride=H * D, q_out=st["q_out"], q_out_stride=Hq * D, slots=st["slots"],
            rows=binding.GEMV_ROWS_F32 if case["rows"] == "f32" else binding.GEMV_ROWS_BF16,
            pairs=binding.GEMV_PAIRS_HALF if case["pairs"] == "half" else binding.GEMV_PAIRS_INTERLEAVED,
            positions=st["positions"], axes=case["axes"], axis_stride=T, freqs=binding.rope_freqs(st["inv"]),
            pair_axis=st["axis"]), cache
    width = st["table"].shape[1]
    if op == "read":
        return binding.gemv_cache_read, binding.cache_read_args(
            table=st["table"], table_width=width, table_stride=width, begin=st["begin"], row_start=st["row_start"],
            requests=case["requests"], rows=st["rows"], k_out=st["outs"]["k"], v_out=st["outs"]["v"],
            k_out_stride=H * D, v_out_stride=H * D,
            row_type=binding.GEMV_ROWS_BF16 if case["out"] == "bf16" else binding.GEMV_ROWS_F32), cache
    Hq = case["q_heads"]
    ws = binding.attn_workspace(Hq, H, D, binding.GEMV_CACHE_FP8_BLOCK, device=DEV)
    return binding.gemv_attn_decode, binding.attn_args(
        q=st["q"], out=st["outs"]["out"], lse=st["outs"].get("lse"), lens=st["lens"], requests=case["requests"],
        q_heads=Hq, q_stride=Hq * D, out_stride=Hq * D, table=st["table"], table_width=width, table_stride=width,
        scale=1.0 / math.sqrt(D), softcap=case["softcap"], window=case["window"], workspace=ws), cache


# ---- plain forms -----------------------------------------------------------

def _rotated(x, st):
    """x [T, H, D] in 32 bits with its first `rot` columns turned by position times frequency, pair by pair."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = st["positions"][st["axis"].long()].double().T * st["inv"]            # [T, half], far angles in 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    x = x.float()
    turned, rest = x[..., :rot], x[..., rot:]
    if case["pairs"] == "half":
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _as_slots(pool, case):
    """A pool as [page, block, slot, head, ...] (codes) or [page, block, head] (scales), whatever its order."""
    if pool.dim() == 3:
        return pool if case["layout"] == "token" else pool.transpose(1, 2)
    pool = pool if case["layout"] == "token" else pool.transpose(1, 2)
    return pool.unflatten(1, (case["page"] // case["block"], case["block"]))


def _write(rows, codes, scales, st):
    """Rows [live, H, D] into their blocks: scales, earlier codes moved with them, the rows' codes."""
    case = st["case"]
    per_page = case["page"] // case["block"]
    page, blk = st["blocks"] // per_page, st["blocks"] % per_page
    NB, H = st["blocks"].numel(), case["kv_heads"]
    top = rows.abs().amax(-1)                                                   # [live, H]
    top = torch.zeros((NB, H), device=DEV).scatter_reduce(0, st["of"][:, None].expand(-1, H), top, "amax")
    m, e = torch.frexp(top)                                                     # top = m 2^e, 1/2 <= m < 1
    need = torch.ldexp(torch.ones_like(top), e - torch.where(m <= 0.875, 9, 8)).clamp(min=SMALLEST)   # 448 = 0.875 * 2^9
    s, c = _as_slots(scales, case), _as_slots(codes.view(torch.uint8), case)
    old = s[page, blk]
    scale = torch.where(st["first"][:, None] > 0, torch.maximum(old, need), need)
    s[page, blk] = scale
    held = c[page, blk]                                                         # [NB, block, H, D]
    moved = (held.view(torch.float8_e4m3fn).float() * (old / scale)[:, None, :, None]).to(torch.float8_e4m3fn)
    before = torch.arange(case["block"], device=DEV)[None, :] < st["first"][:, None]
    c[page, blk] = torch.where(before[:, :, None, None], moved.view(torch.uint8), held)
    slot = st["slots"][:st["live"]].long()
    code = (rows / scale[st["of"]][:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    c[slot // case["page"], slot % case["page"] // case["block"], slot % case["block"]] = code.view(torch.uint8)


def _plain_append(st):
    live = st["live"]
    st["q_out"][:live] = _rotated(st["q"], st)[:live].to(torch.bfloat16)
    _write(_rotated(st["k"], st)[:live], st["kc"], st["ks"], st)
    _write(st["v"][:live].float(), st["vc"], st["vs"], st)
    return st["outs"]


def _gathered(st, n, page):
    """The pages `page` of pool n as values in 32 bits: [..., slot, head, column]."""
    case, kind = st["case"], st["case"].get("kind", "block")
    c = st[n + "c"]
    x = c.view(torch.uint8)[page].view(c.dtype).float() if kind != "bf16" else c[page].float()
    x = x if case["layout"] == "token" else x.transpose(-3, -2)
    if kind == "fp8":
        return x * st[n + "s"][:, None]
    if kind == "bf16":
        return x
    s = st[n + "s"][page]
    s = s if case["layout"] == "token" else s.transpose(-2, -1)
    return x * s.repeat_interleave(case["block"], dim=-2)[..., None]


def _plain_read(st):
    case = st["case"]
    total = st["rows"] - case["pad"]
    row = torch.arange(total, device=DEV)
    r = torch.searchsorted(st["row_start"][1:].long(), row, right=True)
    tok = st["begin"].long()[r] + row - st["row_start"].long()[r]
    page = st["table"][r, tok // case["page"]].long()
    for n in ("k", "v"):
        c, s = st[n + "c"], st.get(n + "s")
        at = (page, tok % case["page"]) if case["layout"] == "token" else (page, slice(None), tok % case["page"])
        x = c[at].float() if case["kind"] == "bf16" else c.view(torch.uint8)[at].view(c.dtype).float()
        if case["kind"] == "fp8":
            x = x * s[:, None]
        elif case["kind"] == "block":
            b = tok % case["page"] // case["block"]
            x = x * (s[page, b] if case["layout"] == "token" else s[page, :, b])[..., None]
        st["outs"][n][:total] = x.to(st["outs"][n].dtype)
    return st["outs"]


def _plain_attn(st):
    """softmax(cap(scale q k)) v over the pages that each request's row of the table names."""
    case = st["case"]
    R, Hq, Hk, D = case["requests"], case["q_heads"], case["kv_heads"], case["dim"]
    lens, table = st["lens"].long(), st["table"].long().clamp(min=0)
    L = table.shape[1] * case["page"]
    at = torch.arange(L, device=DEV)
    seen = at[None, :] < lens[:, None]
    if case["window"]:
        seen = seen & (at[None, :] >= lens[:, None] - case["window"])
    seen = seen[:, None, :, None]

    def rows(n):
        x = _gathered(st, n, table).permute(0, 3, 1, 2, 4)                      # [R, H, W, P, D]
        return x.reshape(R, Hk, L, D).masked_fill(~seen, 0.0)

    s = torch.matmul(st["q"].float().view(R, Hk, Hq // Hk, D), rows("k").transpose(2, 3)) / math.sqrt(D)
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    s = s.masked_fill(~seen.transpose(2, 3), -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows("v")) / total.clamp(min=torch.finfo(torch.float32).tiny)
    st["outs"]["out"].copy_(o.reshape(R, Hq, D))
    if case["lse"]:
        st["outs"]["lse"].copy_(torch.where(total > 0, top + torch.log(total), -math.inf).reshape(R, Hq))
    return st["outs"]


# ---- what a pass cannot do without -----------------------------------------

def _total(lo, hi, n, f=lambda x: x):
    return sum(f(_at(lo, hi, i, n)) for i in range(n))


def work(case):
    op, H, D, P = case["op"], case["kv_heads"], case["dim"], case["page"]
    if op == "append":
        R, Hq = case["requests"], case["q_heads"]
        live = _total(case["new_lo"], case["new_hi"], R)
        blocks = _total(case["new_lo"], case["new_hi"], R, lambda n: -(-n // case["block"]))
        # rows in, q and codes out, positions and slots in, scales in and out (the codes of blocks that grow: not counted)
        return {"bytes": live * D * ((4 if case["rows"] == "f32" else 2) * (Hq + 2 * H) + 2 * Hq + 2 * H)
                + 4 * (live + case["pad"]) * (case["axes"] + 1) + 16 * blocks * H + 8 * case["rot"],
                "flops": 3 * live * (Hq + H) * case["rot"]}
    if op == "read":
        R = case["requests"]
        n = _total(case["lo"], case["hi"], R, lambda x: int(x * case["part"]))
        es, os = 2 if case["kind"] == "bf16" else 1, 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * n * H * (D * (es + os) + (4 / case["block"] if case["kind"] == "block" else 0)) + 4 * n / P + 8 * R,
                "flops": 2 * n * H * D}
    R, Hq = case["requests"], case["q_heads"]
    reach = lambda f: _total(case["lo"], case["hi"], R, lambda n: f(min(n, case["window"] or n)))  # noqa: E731
    seen = reach(lambda n: n)
    return {"bytes": 2 * seen * H * D + 8 * H * reach(lambda n: -(-n // case["block"])) + 4 * reach(lambda n: -(-n // P))
            + 4 * R * Hq * D + 4 * R + (4 * R * Hq if case["lse"] else 0), "flops": 4 * seen * Hq * D}


# ---- from the definition, in 64 bits ---------------------------------------

def exact(case, seed):
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](prepare(case, seed))


def _exact_append(st):
    """Each pair as a complex number times exp(i angle); then block by block, in the order of the batch."""
    case = st["case"]
    half, rot, live, P, B = case["rot"] // 2, case["rot"], st["live"], case["page"], case["block"]
    axis = st["axis"].tolist()
    angles = torch.stack([st["positions"][axis[i]].double() * float(st["inv"][i]) for i in range(half)], 1)
    turn = torch.polar(torch.ones_like(angles), angles)
    first, second = (slice(0, half), slice(half, rot)) if case["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))

    def rotate(x):
        y = x.double().clone()
        z = torch.complex(x[:, :, first].double(), x[:, :, second].double()) * turn[:, None, :]
        y[:, :, first], y[:, :, second] = z.real, z.imag
        return y

    q = st["q_out"].double()
    q[:live] = rotate(st["q"])[:live]
    out = dict(q=q)
    slots = st["slots"][:live].tolist()
    runs, t = [], 0                                             # neighbouring tokens of a block
    while t < live:
        n = 1
        while t + n < live and slots[t + n] // B == slots[t] // B:
            n += 1
        runs.append((t, n))
        t += n
    for name, rows in (("k", rotate(st["k"])), ("v", st["v"].double())):
        codes, scales = st[name + "c"].double(), st[name + "s"].double().clone()
        peak = rows.abs().amax(-1).cpu()
        s_host = scales.cpu()
        for t, n in runs:
            page, place = slots[t] // P, slots[t] % P
            c = codes[page] if case["layout"] == "token" else codes[page].transpose(0, 1)       # [slot, head, column]
            s = s_host[page, place // B] if case["layout"] == "token" else s_host[page, :, place // B]
            need = [max(SMALLEST, 2.0 ** math.ceil(math.log2(x / 448.0))) if x > 0 else SMALLEST
                    for x in peak[t:t + n].amax(0).tolist()]
            old = s.clone()
            s.copy_(torch.tensor(need, dtype=torch.float64) if place % B == 0
                    else torch.maximum(old, torch.tensor(need, dtype=torch.float64)))
            lo = place // B * B
            if place % B:
                c[lo:place] *= (old / s).to(DEV)[:, None]
            c[place:place + n] = (rows[t:t + n] / s.to(DEV)[:, None]).clamp(-448.0, 448.0)
        out[name], out[name + "s"] = codes, s_host.to(DEV)
    return out


def _token_values(st, n, r, begin, end, h):
    """Values of head h of pool n for the tokens begin .. end - 1 of request r, in 64 bits."""
    case, kind = st["case"], st["case"].get("kind", "block")
    P = case["page"]
    pages = st["table"][r, begin // P:-(-end // P)].long()
    c = st[n + "c"][:, :, h] if case["layout"] == "token" else st[n + "c"][:, h]
    x = (c.view(torch.uint8)[pages].view(c.dtype) if kind != "bf16" else c[pages]).double()     # [page, slot, column]
    if kind == "fp8":
        x = x * st[n + "s"][h].double()
    elif kind == "block":
        s = st[n + "s"][:, :, h] if case["layout"] == "token" else st[n + "s"][:, h]
        x = (x.unflatten(1, (P // case["block"], -1)) * s[pages].double()[:, :, None, None]).flatten(1, 2)
    skip = begin % P
    return x.reshape(-1, case["dim"])[skip:skip + end - begin]


def _exact_read(st):
    case = st["case"]
    starts, begin = st["row_start"].tolist(), st["begin"].tolist()
    out = {}
    for n in ("k", "v"):
        y = st["outs"][n].double()
        for r in range(case["requests"]):
            count = starts[r + 1] - starts[r]
            for h in range(case["kv_heads"] if count else 0):
                y[starts[r]:starts[r + 1], h] = _token_values(st, n, r, begin[r], begin[r] + count, h)
        out[n] = y
    return out


def _exact_attn(st):
    case = st["case"]
    R, Hq, Hk, D = case["requests"], case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // Hk
    out = torch.zeros((R, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, n in enumerate(st["lens"].tolist()):
        begin = max(0, n - case["window"]) if case["window"] else 0
        for h in range(Hk if n else 0):
            x = _token_values(st, "k", r, begin, n, h) @ st["q"][r, h * G:(h + 1) * G].double().T * D ** -0.5     # [n, G]
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            z = torch.logsumexp(x, 0)
            lse[r, h * G:(h + 1) * G] = z
            out[r, h * G:(h + 1) * G] = torch.exp(x - z).T @ _token_values(st, "v", r, begin, n, h)
    return dict(out=out, lse=lse) if case["lse"] else dict(out=out)
