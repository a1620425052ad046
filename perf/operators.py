"""The attention half of a decode step, as cases: page bookkeeping, rotary
positions with the cache write, and attention of one new token over the paged
key-value cache. Each case runs either in its plain form (elementary torch
operations in 32 bits, or in 64 where 32 lose what matters) or, with ``own``
true, through the entry points of the package's binding.

Head counts, head size and page tables follow the decode step of this package
(32 query heads, 8 key-value heads, 128 columns a head); the others are generic.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # One decode step of a batch: every request gets one token, some of them a new page.
        dict(name="tables-decode", op="tables", requests=64, lo=1, hi=4096, new_lo=1, new_hi=1,
             page=16, width=512, spare=128, room=64),
        # A batch of prompts next to requests that wait, into a pool that runs out for the last ones.
        dict(name="tables-prompts", op="tables", requests=509, lo=0, hi=1500, new_lo=0, new_hi=2047,
             page=32, width=256, spare=15000, room=530000),
        # The new token of 16 requests: FP32 projections in, far positions, BF16 cache.
        dict(name="rope-append-decode", op="append", tokens=16, pad=0, q_heads=32, kv_heads=8, dim=128, rot=128,
             axes=1, pairs="half", rows="f32", kind="bf16", layout="token", page=16, pages=64, far=131072),
        # A prompt of 4,096 tokens, a ragged end of padding rows.
        dict(name="rope-append-prompt", op="append", tokens=4096, pad=33, q_heads=32, kv_heads=8, dim=128, rot=128,
             axes=1, pairs="half", rows="f32", kind="bf16", layout="head", page=32, pages=160, far=8192),
        # Image and text tokens with three axes of positions, into an FP8 cache.
        dict(name="rope-append-fp8-axes", op="append", tokens=1021, pad=5, q_heads=32, kv_heads=8, dim=128, rot=128,
             axes=3, pairs="half", rows="bf16", kind="fp8", layout="head", page=64, pages=20, far=32768),
        # Image patches with two axes, no cache, heads of 80 columns.
        dict(name="rope-image", op="rope", tokens=8100, pad=0, q_heads=16, kv_heads=16, dim=80, rot=80,
             axes=2, pairs="interleaved", rows="bf16", far=128),
        # The latency of one request with a short context.
        dict(name="attn-1x1000", op="attn", requests=1, lo=1000, hi=1000, q_heads=32, kv_heads=8, dim=128,
             kind="bf16", layout="token", page=16, window=0, softcap=0.0, lse=True),
        # An ordinary batch with contexts of all lengths, a request without any among them.
        dict(name="attn-16x4k", op="attn", requests=16, lo=0, hi=4096, q_heads=32, kv_heads=8, dim=128,
             kind="bf16", layout="token", page=16, window=0, softcap=0.0, lse=False),
        # A large batch with long contexts.
        dict(name="attn-64x32k", op="attn", requests=64, lo=16384, hi=32768, q_heads=32, kv_heads=8, dim=128,
             kind="bf16", layout="token", page=64, window=0, softcap=0.0, lse=False),
        # FP8 cache, contexts of up to 16,384 tokens.
        dict(name="attn-32x16k-fp8", op="attn", requests=32, lo=37, hi=16384, q_heads=32, kv_heads=8, dim=128,
             kind="fp8", layout="head", page=32, window=0, softcap=0.0, lse=True),
        # One request with a very long context: nothing but the split over its length fills the GPU.
        dict(name="attn-1x131072", op="attn", requests=1, lo=131071, hi=131071, q_heads=32, kv_heads=8, dim=128,
             kind="bf16", layout="head", page=64, window=0, softcap=0.0, lse=False),
        # Wide heads in groups of 16, a sliding window and capped scores, pages that divide no tile.
        dict(name="attn-wide-window", op="attn", requests=48, lo=0, hi=9000, q_heads=32, kv_heads=2, dim=256,
             kind="bf16", layout="head", page=24, window=4096, softcap=50.0, lse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "rope", "attn", "attn", "attn", "attn"])
    if op == "tables":
        requests, page = _log_int(rng, 1, 2048), rng.choice([1, 7, 16, 24, 32, 64, 128])
        hi, new_hi = _log_int(rng, 1, 8192), rng.choice([1, 1, _log_int(rng, 2, 2048)])
        while requests * new_hi > 1_000_000:
            new_hi = max(1, new_hi // 2)
        need = requests * (new_hi // (2 * page) + 1)
        return dict(op=op, requests=requests, lo=rng.choice([0, 1]), hi=hi, new_lo=rng.choice([0, 1]), new_hi=new_hi,
                    page=page, width=max(-(-hi // page), (hi + new_hi) // page + rng.choice([0, 1, 9])),
                    spare=max(1, int(need * rng.choice([0.4, 1.2, 2.5]))),
                    room=max(1, int(requests * (new_hi + 1) * rng.choice([0.45, 0.6, 1.0]))))
    if op in ("append", "rope"):
        dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        q_heads = kv_heads * rng.choice([1, 2, 4, 4, 7, 8])
        most = 4096 * 48 * 128 // ((q_heads + 2 * kv_heads) * dim)
        tokens = _log_int(rng, 1, max(2, min(8192, most)))
        case = dict(op=op, tokens=tokens, pad=rng.choice([0, 0, tokens // 9]), q_heads=q_heads, kv_heads=kv_heads,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 2, 3]),
                    pairs=rng.choice(["half", "half", "interleaved"]), rows=rng.choice(["f32", "bf16"]),
                    far=_log_int(rng, 2, 1 << 20))
        if op == "append":
            page = rng.choice([1, 8, 16, 24, 32, 64])
            case.update(kind=rng.choice(["bf16", "fp8"]), layout=rng.choice(["token", "head"]), page=page,
                        pages=tokens // page + rng.choice([1, 2, 5]))
        return case
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8, 16, 32])
    requests, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
    while requests * hi * kv_heads * dim > 64 * 24000 * 8 * 128:
        requests, hi = max(1, requests * 3 // 4), max(1, hi * 3 // 4)
    return dict(op=op, requests=requests, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, kind=rng.choice(["bf16", "bf16", "fp8"]),
                layout=rng.choice(["token", "head"]), page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]),
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]), softcap=rng.choice([0.0, 0.0, 30.0]),
                lse=rng.choice([True, False]))


# ---- inputs ----------------------------------------------------------------

def _spaced(lo, hi, n, g):
    """n whole numbers from lo to hi, evenly spaced, in an order of the seed's: the same sum for every seed."""
    v = torch.tensor([hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)], dtype=torch.int64)
    return v[torch.randperm(n, generator=g)]


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_rope, "rope": _prepare_rope,
            "attn": _prepare_attn}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    g = _gen(seed, "cpu")
    R, P, W = case["requests"], case["page"], case["width"]
    lens = _spaced(case["lo"], case["hi"], R, g)
    new = _spaced(case["new_lo"], case["new_hi"], R, g)
    have = (lens + P - 1) // P
    held = int(have.sum())
    num_pages = held + case["spare"]
    order = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((R + 1, W), -1, dtype=torch.int32)      # one more row than requests: the plain form's spill
    at = torch.arange(W)
    mine = at[None, :] < have[:, None]
    table[:R][mine] = order[:held]
    taken = int(torch.randint(0, 4, (1,), generator=g))        # pages of the list that earlier steps took
    free = torch.cat([torch.zeros(taken, dtype=torch.int32), order[held:]])
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, R=R, num_pages=num_pages, table=table.to(DEV), lens=lens.to(**i32), new=new.to(**i32),
                free=free.to(DEV), free_next=torch.tensor([taken], **i32),
                slots=torch.empty(case["room"], **i32), positions=torch.empty(case["room"], **i32),
                token_start=torch.empty(R + 1, **i32), page_start=torch.empty(R, **i32),
                new_lens=torch.empty(R, **i32), status=torch.empty(R, **i32), free_next_out=torch.empty(1, **i32))


def _inv_freq(case):
    """base^(-2i / rot) for pair i, and the axis of pair i: equal shares of the pairs, the first axis's first."""
    half = case["rot"] // 2
    inv = torch.tensor([500000.0 ** (-2.0 * i / case["rot"]) for i in range(half)], dtype=torch.float64)
    axis = torch.tensor([min(i * case["axes"] // half, case["axes"] - 1) for i in range(half)], dtype=torch.int32)
    return inv, axis


def _prepare_rope(case, seed):
    g = _gen(seed, DEV)
    T, Hq, Hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    dt = torch.float32 if case["rows"] == "f32" else torch.bfloat16
    r = lambda *s, d=dt: torch.randn(s, generator=g, device=DEV, dtype=d)  # noqa: E731
    inv, axis = _inv_freq(case)
    st = dict(case=case, q=r(T, Hq, D), k=r(T, Hk, D), inv=inv.to(DEV), axis=axis.to(DEV),
              positions=torch.randint(0, case["far"], (case["axes"], T), generator=g, device=DEV, dtype=torch.int32),
              q_out=r(T, Hq, D, d=torch.bfloat16))
    if case["op"] == "rope":
        st["k_out"] = r(T, Hk, D, d=torch.bfloat16)
        return st
    pages, P = case["pages"], case["page"]
    st["v"] = r(T, Hk, D)
    shape = (pages + 1, P, Hk, D) if case["layout"] == "token" else (pages + 1, Hk, P, D)   # a page more: see _put
    for n in ("kc", "vc"):
        st[n] = r(*shape, d=torch.bfloat16)
        if case["kind"] == "fp8":
            st[n] = st[n].to(torch.float8_e4m3fn)
    if case["kind"] == "fp8":
        st["ks"] = 2.0 ** torch.randint(-6, -3, (Hk,), generator=g, device=DEV).float()
        st["vs"] = 2.0 ** torch.randint(-6, -3, (Hk,), generator=g, device=DEV).float()
    slots = torch.randperm(pages * P, generator=g, device=DEV)[:T].to(torch.int32)
    slots[T - case["pad"]:] = -1                                  # rows behind the last sequence
    st["slots"] = slots
    return st


def _prepare_attn(case, seed):
    g, gc = _gen(seed, DEV), _gen(seed, "cpu")
    R, Hq, Hk, D, P = case["requests"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _spaced(case["lo"], case["hi"], R, gc)
    have = (lens + P - 1) // P
    held = int(have.sum())
    num_pages = held + 3
    W = max(1, -(-case["hi"] // P))
    order = torch.randperm(num_pages, generator=gc).to(torch.int32)
    table = torch.full((R, W), -1, dtype=torch.int32)
    table[torch.arange(W)[None, :] < have[:, None]] = order[:held]
    shape = (num_pages, P, Hk, D) if case["layout"] == "token" else (num_pages, Hk, P, D)
    st = dict(case=case, lens=lens.to(DEV, torch.int32), table=table.to(DEV), num_pages=num_pages,
              q=2 * torch.randn((R, Hq, D), generator=g, device=DEV, dtype=torch.bfloat16))
    for n in ("kc", "vc"):
        st[n] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        if case["kind"] == "fp8":
            st[n] = (st[n] * 32).to(torch.float8_e4m3fn)
    if case["kind"] == "fp8":
        st["ks"] = (torch.rand(Hk, generator=g, device=DEV) + 0.5) / 32
        st["vs"] = (torch.rand(Hk, generator=g, device=DEV) + 0.5) / 32
    st["out"] = torch.empty((R, Hq, D), device=DEV, dtype=torch.bfloat16)
    st["lse"] = torch.empty((R, Hq), device=DEV, dtype=torch.float32) if case["lse"] else None
    return st


# ---- one pass --------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "append": _plain_append, "rope": _plain_rope,
            "attn": _plain_attn}[state["case"]["op"]](state)


def _own(st):
    """The package's calls. The argument records name buffers, as a serving loop's do, and are filled once."""
    from memory_bound_decode_gb300 import binding
    case, op = st["case"], st["case"]["op"]
    if "args" not in st:
        st["args"], st["cache"] = _records(binding, st)
    if op == "tables":
        binding.gemv_block_tables(st["args"])
        return dict(table=st["table"][:st["R"]], slots=st["slots"], positions=st["positions"],
                    token_start=st["token_start"], page_start=st["page_start"], new_lens=st["new_lens"],
                    status=st["status"], free_next=st["free_next_out"])
    if op == "rope":
        binding.gemv_rope(st["args"])
        return dict(q=st["q_out"], k=st["k_out"])
    if op == "append":
        binding.gemv_rope_append(st["args"], st["cache"])
        return dict(q=st["q_out"], k=st["kc"][:case["pages"]], v=st["vc"][:case["pages"]])
    binding.gemv_attn_decode(st["args"], st["cache"])
    return dict(out=st["out"], lse=st["lse"]) if case["lse"] else dict(out=st["out"])


def _records(binding, st):
    case, op = st["case"], st["case"]["op"]
    if op == "tables":
        return binding.block_tables_args(
            lens=st["lens"], new_tokens=st["new"], requests=st["R"], page_size=case["page"],
            num_pages=st["num_pages"], table=st["table"], table_width=case["width"], table_stride=case["width"],
            free_pages=st["free"], free_cap=st["free"].numel(), free_next=st["free_next"],
            max_tokens=case["room"], slots=st["slots"], positions=st["positions"], token_start=st["token_start"],
            page_start=st["page_start"], new_lens=st["new_lens"], status=st["status"],
            free_next_out=st["free_next_out"]), None
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["dim"]
    cache = None
    if op in ("append", "attn"):
        P = case["page"]
        slot, head = (Hk * D, D) if case["layout"] == "token" else (D, P * D)
        cache = binding.kv_cache(
            st["kc"], st["vc"], num_pages=st["num_pages"] if op == "attn" else case["pages"], page_size=P,
            kv_heads=Hk, head_dim=D, page_stride=P * Hk * D, head_stride=head, slot_stride=slot,
            kind=binding.GEMV_CACHE_FP8 if case["kind"] == "fp8" else binding.GEMV_CACHE_BF16,
            k_scale=st.get("ks"), v_scale=st.get("vs"))
    if op == "attn":
        ws = binding.attn_workspace(Hq, Hk, D, device=DEV)
        return binding.attn_args(
            q=st["q"], out=st["out"], lse=st["lse"], lens=st["lens"], requests=case["requests"], q_heads=Hq,
            q_stride=Hq * D, out_stride=Hq * D, table=st["table"], table_width=st["table"].shape[1],
            table_stride=st["table"].shape[1], scale=1.0 / math.sqrt(D), softcap=case["softcap"],
            window=case["window"], workspace=ws), cache
    return binding.rope_args(
        q=st["q"], k=st["k"], v=st.get("v"), tokens=case["tokens"], q_heads=Hq, kv_heads=Hk, head_dim=D,
        rot_dim=case["rot"], q_stride=Hq * D, k_stride=Hk * D, v_stride=Hk * D,
        rows=binding.GEMV_ROWS_F32 if case["rows"] == "f32" else binding.GEMV_ROWS_BF16,
        pairs=binding.GEMV_PAIRS_HALF if case["pairs"] == "half" else binding.GEMV_PAIRS_INTERLEAVED,
        positions=st["positions"], axes=case["axes"], axis_stride=case["tokens"],
        freqs=binding.rope_freqs(st["inv"]), pair_axis=st["axis"], q_out=st["q_out"], q_out_stride=Hq * D,
        k_out=st.get("k_out"), k_out_stride=Hk * D, slots=st.get("slots")), cache


# ---- plain forms -----------------------------------------------------------

def _plain_tables(st):
    """Pages and slots of this step's tokens: running sums over the requests, then every token on its own."""
    case, R = st["case"], st["R"]
    P, W, room, pool = case["page"], case["width"], case["room"], st["num_pages"]
    lens, new, table, free = st["lens"].long(), st["new"].long(), st["table"], st["free"].long()
    count = new.clamp(min=0)
    end = torch.cumsum(count, 0)
    start = end - count
    bad = (lens < 0) | (new < 0)
    long = ~bad & (lens + new > W * P)
    over = ~bad & ~long & (count > 0) & (end > room)
    fits = ~(bad | long | over)
    have = (lens.clamp(min=0) + P - 1) // P
    need = torch.where(fits, (lens + new + P - 1) // P - have, 0)
    page_end = torch.cumsum(need, 0)
    first = st["free_next"].long()
    avail = torch.where(first < 0, 0, (free.numel() - first).clamp(min=0))
    dry = fits & (need > 0) & (page_end > avail)
    served = fits & ~dry
    page_start = first + page_end - need

    t = torch.arange(room, device=lens.device)
    r = torch.searchsorted(end, t, right=True).clamp(max=R - 1)
    live = (t < end[-1]) & served[r]
    pos = lens[r] + t - start[r]
    blk = torch.where(live, pos // P, 0)
    fresh = live & (blk >= have[r])
    taken = free[(page_start[r] + blk - have[r]).clamp(0, free.numel() - 1)]
    page = torch.where(fresh, taken, table[r, blk].long())
    table.index_put_((torch.where(fresh, r, R), torch.where(fresh, blk, 0)), page.to(torch.int32))
    live_slot = live & (page >= 0) & (page < pool)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(table=table[:R], slots=i32(torch.where(live_slot, page * P + pos % P, -1)),
                positions=i32(torch.where(live, pos, 0)),
                token_start=i32(torch.cat([start, end[-1:]]).clamp(max=2 ** 31 - 1)),
                page_start=i32(torch.where(served, page_start, -1)),
                new_lens=i32(torch.where(served, lens + new, lens)),
                status=i32(torch.where(bad, 4, torch.where(long, 2, torch.where(over, 3, torch.where(dry, 1, 0))))),
                free_next=i32(first + torch.where(served, need, 0).sum()))


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


def _plain_rope(st):
    st["q_out"].copy_(_rotated(st["q"], st))
    st["k_out"].copy_(_rotated(st["k"], st))
    return dict(q=st["q_out"], k=st["k_out"])


def _put(cache, rows, scale, st):
    """Rows [T, H, D] at their slots. Rows without a slot go to the page behind the pool's last one."""
    case = st["case"]
    P, slots = case["page"], st["slots"].long()
    page = torch.where(slots < 0, case["pages"], slots // P)
    off = torch.where(slots < 0, 0, slots % P)
    if case["kind"] == "fp8":
        rows = (rows / scale[None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        view = cache.view(torch.uint8)
    else:
        rows, view = rows.to(torch.bfloat16), cache
    (view if case["layout"] == "token" else view.transpose(1, 2)).index_put_((page, off), rows)
    return cache[:case["pages"]]


def _plain_append(st):
    live = (st["slots"] >= 0)[:, None, None]
    st["q_out"].copy_(torch.where(live, _rotated(st["q"], st).to(torch.bfloat16), st["q_out"]))
    return dict(q=st["q_out"], k=_put(st["kc"], _rotated(st["k"], st), st.get("ks"), st),
                v=_put(st["vc"], st["v"].float(), st.get("vs"), st))


def _plain_attn(st):
    """softmax(cap(scale q k)) v over the pages that each request's row of the table names."""
    case = st["case"]
    R, Hq, Hk, D = case["requests"], case["q_heads"], case["kv_heads"], case["dim"]
    lens, table = st["lens"].long(), st["table"].long().clamp(min=0)
    L = table.shape[1] * case["page"]
    at = torch.arange(L, device=lens.device)
    seen = at[None, :] < lens[:, None]
    if case["window"]:
        seen = seen & (at[None, :] >= lens[:, None] - case["window"])
    seen = seen[:, None, :, None]

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[table].view(cache.dtype) if case["kind"] == "fp8" else cache[table]
        x = x.float()                                         # [R, W, P, H, D] or [R, W, H, P, D]
        x = x.permute(0, 3, 1, 2, 4) if case["layout"] == "token" else x.permute(0, 2, 1, 3, 4)
        x = x.reshape(R, Hk, L, D)
        if scale is not None:
            x = x * scale[None, :, None, None]
        return x.masked_fill(~seen, 0.0)

    q = st["q"].float().view(R, Hk, Hq // Hk, D)
    s = torch.matmul(q, gathered(st["kc"], st.get("ks")).transpose(2, 3)) / math.sqrt(D)
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    s = s.masked_fill(~seen.transpose(2, 3), -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gathered(st["vc"], st.get("vs"))) / total.clamp(min=torch.finfo(torch.float32).tiny)
    out = o.reshape(R, Hq, D).to(torch.bfloat16)
    if not case["lse"]:
        return dict(out=out)
    return dict(out=out, lse=torch.where(total > 0, top + torch.log(total), -math.inf).reshape(R, Hq))


# ---- what a pass cannot do without -----------------------------------------

def _totals(lo, hi, n, f=lambda x: x):
    return sum(f(hi if n == 1 else lo + (hi - lo) * i // (n - 1)) for i in range(n))


def work(case):
    op = case["op"]
    if op == "tables":
        R, P = case["requests"], case["page"]
        tokens = min(case["room"], _totals(case["new_lo"], case["new_hi"], R))
        pages = min(case["spare"], tokens // P + R)
        # lengths and counts in, free pages in and table entries out, slots and positions out for every row of the
        # room, per request: first token, first page, length and status
        return {"bytes": 8 * R + 8 * pages + 8 * case["room"] + 16 * R + 12, "flops": 0}
    if op in ("append", "rope"):
        T, Hq, Hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        live = T - case["pad"]
        rows = 4 if case["rows"] == "f32" else 2
        kv = 2 if op == "rope" else 2 * (1 if case["kind"] == "fp8" else 2)
        ins = Hq + (Hk if op == "rope" else 2 * Hk)
        turned = (Hq + Hk) * case["rot"]
        return {"bytes": live * D * (rows * ins + 2 * Hq + kv * Hk) + 4 * T * (case["axes"] + (op == "append"))
                + 8 * case["rot"], "flops": 3 * live * turned}
    R, Hq, Hk, D = case["requests"], case["q_heads"], case["kv_heads"], case["dim"]
    seen = _totals(case["lo"], case["hi"], R, lambda n: min(n, case["window"] or n))
    es = 1 if case["kind"] == "fp8" else 2
    pages = _totals(case["lo"], case["hi"], R, lambda n: -(-min(n, case["window"] or n) // case["page"]))
    return {"bytes": 2 * seen * Hk * D * es + 4 * R * Hq * D + 4 * pages + 4 * R + (4 * R * Hq if case["lse"] else 0),
            "flops": 4 * seen * Hq * D}


# ---- from the definition, in 64 bits ---------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None                                           # whole numbers only
    st = prepare(case, seed)
    return _exact_attn(st) if case["op"] == "attn" else _exact_rope(st)


def _exact_rope(st):
    """Each pair as a complex number times exp(i angle)."""
    case = st["case"]
    half, rot = case["rot"] // 2, case["rot"]
    axis = st["axis"].tolist()
    angles = torch.stack([st["positions"][axis[i]].double() * float(st["inv"][i]) for i in range(half)], 1)
    turn = torch.polar(torch.ones_like(angles), angles)
    if case["pairs"] == "half":
        first, second = list(range(half)), list(range(half, rot))
    else:
        first, second = list(range(0, rot, 2)), list(range(1, rot, 2))

    def rotate(x):
        y = x.double().clone()
        z = torch.complex(x[:, :, first].double(), x[:, :, second].double()) * turn[:, None, :]
        y[:, :, first], y[:, :, second] = z.real, z.imag
        return y

    live = torch.nonzero(st["slots"] >= 0).flatten() if case["op"] == "append" else torch.arange(case["tokens"], device=DEV)
    q = st["q_out"].double()
    q[live] = rotate(st["q"])[live]
    if case["op"] == "rope":
        return dict(q=q, k=rotate(st["k"]))
    slot = st["slots"].long()[live]
    out = dict(q=q)
    for name, rows, scale in (("k", rotate(st["k"]), "ks"), ("v", st["v"].double(), "vs")):
        c = st[name + "c"][:case["pages"]].double()
        rows = rows[live]
        if case["kind"] == "fp8":
            rows = torch.clamp(rows / st[scale].double()[:, None], -448, 448)
        if case["layout"] == "token":
            c.view(-1, *c.shape[2:])[slot] = rows
        else:
            c[slot // case["page"], :, slot % case["page"], :] = rows
        out[name] = c
    return out


def _exact_attn(st):
    case = st["case"]
    R, Hq, Hk, D, P = case["requests"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    G = Hq // Hk
    out = torch.zeros((R, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        pages = st["table"][r, :-(-n // P)].long()
        begin = max(0, n - case["window"]) if case["window"] else 0
        for h in range(Hk):
            def rows(cache, scale):
                c = (cache[:, :, h] if case["layout"] == "token" else cache[:, h])
                c = c.view(torch.uint8)[pages].view(c.dtype) if case["kind"] == "fp8" else c[pages]
                c = c.reshape(-1, D)[begin:n].double()
                return c * scale[h].double() if scale is not None else c
            x = rows(st["kc"], st.get("ks")) @ st["q"][r, h * G:(h + 1) * G].double().T * D ** -0.5    # [n, G]
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            z = torch.logsumexp(x, 0)
            lse[r, h * G:(h + 1) * G] = z
            out[r, h * G:(h + 1) * G] = torch.exp(x - z).T @ rows(st["vc"], st.get("vs"))
    return dict(out=out, lse=lse) if case["lse"] else dict(out=out)
