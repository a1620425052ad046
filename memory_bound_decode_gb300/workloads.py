"""Decode-projection workloads: shapes of a Llama-3.1-8B-shaped model (random
init, shapes only) and the device-resident decode step built from them.

One decode step at batch 1 multiplies, in every layer, the hidden vector by the
fused Q/K/V projection (4,096 + 1,024 + 1,024 rows), the output projection
(4,096 rows), the fused gate/up projection (14,336 + 14,336 rows) and the down
projection (4,096 rows over K = 14,336), then the LM head (128,256 rows)
("Decode GEMV at half of HBM bandwidth", causes 1 and 3; "GPU performance
chains", "Launch gaps in a decode step"). The projections are not chained: with
random weights and no nonlinearity in between, each layer reads its own
activation vector x4096_l (shared by QKV, o_proj and gate/up) and x14336_l
(read by down); the LM head reads its own x. Each projection group is one
launch: 4 per layer plus the LM head, 129 for 32 layers, captured as one graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding, inputs, roofline

LLAMA_8B = dict(layers=32, hidden=4096, intermediate=14336, vocab=128256, q_rows=4096, kv_rows=1024)

# Single-projection shapes (N, K) of that model.
SHAPES = {
    "k_proj": (1024, 4096),
    "down_proj": (4096, 14336),
    "qkv": (6144, 4096),
    "o_proj": (4096, 4096),
    "gate_up": (28672, 4096),
    "lm_head": (128256, 4096),
}

# Ragged shapes with ldw = K rounded up to a multiple of 8.
TAILS = [(7, 129), (4097, 4103), (1, 8191), (33, 65537)]


def decode_step_spec(**overrides) -> dict:
    spec = dict(LLAMA_8B)
    spec.update(overrides)
    return spec


@dataclass
class Proj:
    name: str
    W: torch.Tensor          # BF16 weights, or the INT4 / FP8 codes
    x: torch.Tensor
    y: torch.Tensor
    N: int
    K: int
    ldw: int                 # row stride (elements for BF16, bytes for codes)
    group: int
    S: torch.Tensor | None = None   # INT4 group scales / FP8 row scales
    lds: int = 0


WEIGHT_KINDS = {"bf16": binding.GEMV_WEIGHT_BF16, "int4": binding.GEMV_WEIGHT_INT4,
                "fp8": binding.GEMV_WEIGHT_FP8}


class DecodeStep:
    """Device-resident weights, activations and outputs of one decode step, with
    BF16, INT4 (128-column groups, BF16 scales) or FP8 (E4M3, FP32 row scales)
    weights."""

    def __init__(self, spec: dict, seed: int = 0, device="cuda", weights: str = "bf16", batch: int = 1):
        if weights not in WEIGHT_KINDS:
            raise ValueError(f"weights must be one of {sorted(WEIGHT_KINDS)}")
        if not 1 <= batch <= binding.GEMV_MAX_BATCH:
            raise ValueError("batch must be 1..16")
        self.spec = spec
        self.device = device
        self.weights = weights
        self.batch = batch
        self.projs: list[Proj] = []
        self.xs: list[tuple[torch.Tensor, int]] = []
        H, I, V = spec["hidden"], spec["intermediate"], spec["vocab"]
        Q, KV = spec["q_rows"], spec["kv_rows"]
        L = spec["layers"]
        # Every activation vector lives in one buffer and every output in
        # another (views at 16-byte multiples), so a step's inputs and outputs
        # each cross the host link as one copy (gemv_plan_launch_host_io).
        self.x_arena = torch.empty(batch * (L * (H + I) + H), dtype=torch.bfloat16, device=device)
        self.y_arena = torch.empty(batch * (L * (Q + 2 * KV + H + 2 * I + H) + V), dtype=torch.float32,
                                   device=device)
        self._x_off = 0
        self._y_off = 0
        group = 0
        for l in range(spec["layers"]):
            base = 16 * l
            xh = self._x_view(inputs.activations(batch, H, seed=seed, index=base + 14, device=device))
            xi = self._x_view(inputs.activations(batch, I, seed=seed, index=base + 15, device=device))
            self.xs += [(xh, base + 14), (xi, base + 15)]
            group += 1
            for j, (nm, n) in enumerate([("q", Q), ("k", KV), ("v", KV)]):
                self._add(f"l{l}.{nm}_proj", n, H, xh, group, seed, base + j)
            self._add(f"l{l}.o_proj", H, H, xh, 0, seed, base + 3)
            group += 1
            self._add(f"l{l}.gate_proj", I, H, xh, group, seed, base + 4)
            self._add(f"l{l}.up_proj", I, H, xh, group, seed, base + 5)
            self._add(f"l{l}.down_proj", H, I, xi, 0, seed, base + 6)
        base = 16 * spec["layers"]
        xl = self._x_view(inputs.activations(batch, H, seed=seed, index=base + 1, device=device))
        self.xs.append((xl, base + 1))
        self._add("lm_head", V, H, xl, 0, seed, base)
        assert self._x_off == self.x_arena.numel() and self._y_off == self.y_arena.numel()

    def _x_view(self, x: torch.Tensor) -> torch.Tensor:
        B, n = x.shape
        v = self.x_arena[self._x_off:self._x_off + B * n].view(B, n)
        v.copy_(x)
        self._x_off += B * n
        return v

    def _add(self, name, N, K, x, group, seed, index):
        y = self.y_arena[self._y_off:self._y_off + self.batch * N].view(self.batch, N)
        self._y_off += self.batch * N
        if self.weights == "bf16":
            ldw = inputs.padded_ldw(K)
            W = inputs.weight(N, K, ldw, seed=seed, index=index, device=self.device)
            self.projs.append(Proj(name, W, x, y, N, K, ldw, group))
        elif self.weights == "fp8":
            W, S = inputs.fp8_weight(N, K, seed=seed, index=index, device=self.device)
            self.projs.append(Proj(name, W, x, y, N, K, W.shape[1], group, S, 0))
        else:
            W, S = inputs.w4_weight_device(N, K, seed=seed, index=index, device=self.device)
            self.projs.append(Proj(name, W, x, y, N, K, W.shape[1], group, S, S.shape[1]))

    def plan(self, rms_eps: float | None = None, streamk: bool = False) -> binding.Plan:
        """The step as one plan. With rms_eps, the projections that read a
        normalised activation in the model (QKV, gate/up and the LM head) take
        the RMSNorm prologue; o_proj and down read the raw one. With streamk,
        every launch runs the stream-K kernel."""
        def eps_of(p):
            if rms_eps is None:
                return None
            return rms_eps if (p.name.endswith(("q_proj", "k_proj", "v_proj", "gate_proj", "up_proj"))
                               or p.name == "lm_head") else None
        kind = WEIGHT_KINDS[self.weights]
        return binding.Plan([(p.W, p.x, p.y, p.N, p.K, p.ldw, self.batch, p.group, eps_of(p), streamk, kind, p.S,
                              p.lds) for p in self.projs], keepalive=self)

    def outputs(self):
        return [p.y for p in self.projs]

    def refresh_x(self, seed: int) -> None:
        """Overwrite every activation vector in place (the plan keeps its addresses)."""
        for x, index in self.xs:
            x.copy_(inputs.activations(self.batch, x.shape[1], seed=seed, index=index, device=self.device))

    def checks(self):
        for p in self.projs:
            yield p.name, p.W, p.x, p.y, p.K

    def _wbytes(self, p) -> int:
        """Weight bytes of one projection: BF16 2*N*K; INT4 N*K/2 codes plus
        2*N*K/128 scale bytes; FP8 N*K codes plus 4*N scale bytes."""
        if self.weights == "bf16":
            return 2 * p.N * p.K
        if self.weights == "fp8":
            return p.N * p.K + 4 * p.N
        return p.N * p.K // 2 + 2 * p.N * (p.K // inputs.W4_GROUP)

    def algorithmic_bytes(self) -> int:
        """Sum of weight bytes + B*K*2 + B*N*4 over the projections; a fused
        launch moves its x once, so each launch group counts x once."""
        total = 0
        seen_groups = set()
        for p in self.projs:
            total += self._wbytes(p) + 4 * self.batch * p.N
            if p.group == 0 or p.group not in seen_groups:
                total += 2 * self.batch * p.K
                seen_groups.add(p.group)
        return total

    def weight_bytes(self) -> int:
        return sum(self._wbytes(p) for p in self.projs)


def step_bytes_formula(spec: dict, batch: int = 1) -> int:
    """Algorithmic bytes of the step at `batch` rows of x, with fused groups
    counted as one GEMV each (QKV 6,144 rows; gate/up 28,672 rows)."""
    H, I, V = spec["hidden"], spec["intermediate"], spec["vocab"]
    Q, KV = spec["q_rows"], spec["kv_rows"]
    B = batch
    layer = (roofline.algorithmic_bytes(Q + 2 * KV, H, B) + roofline.algorithmic_bytes(H, H, B)
             + roofline.algorithmic_bytes(2 * I, H, B) + roofline.algorithmic_bytes(H, I, B))
    return spec["layers"] * layer + roofline.algorithmic_bytes(V, H, B)


class AttentionStep:
    """The attention half of a decode step, chained and captured: per layer the
    fused Q/K/V projection, rotary positions with the cache write, attention of
    the new token over the paged cache, and the output projection, behind one
    call that gives the batch's new tokens their pages and slots. The layers'
    inputs are not chained (as in DecodeStep): each reads its own x.

    ``context``: tokens each request holds already (an int, or one per request).
    With ``advance`` every step appends a token (lengths and the place in the
    free list move on in place, so a replayed graph is one step after the
    other), for up to ``room`` steps; without, every step writes the same token
    again. ``cache``: "bf16", "fp8" (E4M3, a scale per key-value head) or "fp8_block" (E4M3, a scale for each block of
    tokens, a page or a part of one, and key-value head, found as they are written).
    """

    def __init__(self, spec: dict, context, batch: int = 1, seed: int = 0, device="cuda", cache: str = "bf16",
                 head_dim: int = 128, page_size: int = 16, advance: bool = False, room: int = 64,
                 rope_base: float = 500000.0):
        if not 1 <= batch <= binding.GEMV_MAX_BATCH:
            raise ValueError("batch must be 1..16")
        if cache not in ("bf16", "fp8", "fp8_block"):
            raise ValueError("cache must be bf16, fp8 or fp8_block")
        lens = [context] * batch if isinstance(context, int) else list(context)
        if len(lens) != batch or min(lens) < 0:
            raise ValueError("context must be a length, or one per request")
        self.spec, self.batch, self.cache, self.head_dim, self.page_size = spec, batch, cache, head_dim, page_size
        self.context, self.advance, self.device = lens, advance, device
        H, Q, KV = spec["hidden"], spec["q_rows"], spec["kv_rows"]
        if Q % head_dim or KV % head_dim:
            raise ValueError("q_rows and kv_rows must be whole heads")
        self.q_heads, self.kv_heads = Q // head_dim, KV // head_dim
        self.ldw_h, self.ldw_q = inputs.padded_ldw(H), inputs.padded_ldw(Q)
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        # Pages: what the requests hold, then room for the steps, in a shuffled order.
        have = [-(-n // page_size) for n in lens]
        self.width = max(-(-(n + room) // page_size) for n in lens)
        spare = sum(-(-(n + room) // page_size) for n in lens) - sum(have)
        self.num_pages = sum(have) + spare
        order = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((batch, self.width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(have):
            table[r, :n] = order[at:at + n]
            at += n
        i32 = dict(dtype=torch.int32, device=device)
        self.table = table.to(device)
        self.free = order[at:].contiguous().to(device)
        self.free_next = torch.zeros(1, **i32)
        self.lens = torch.tensor(lens, **i32)
        self.new_lens = self.lens if advance else torch.empty(batch, **i32)
        free_next_out = self.free_next if advance else torch.empty(1, **i32)
        self.ones = torch.ones(batch, **i32)
        self.slots, self.positions, self.page_start, self.status = (torch.empty(batch, **i32) for _ in range(4))
        self.token_start = torch.empty(batch + 1, **i32)
        self.tables = binding.block_tables_args(
            lens=self.lens, new_tokens=self.ones, requests=batch, page_size=page_size, num_pages=self.num_pages,
            table=self.table, table_width=self.width, table_stride=self.width, free_pages=self.free,
            free_cap=self.free.numel(), free_next=self.free_next, max_tokens=batch, slots=self.slots,
            positions=self.positions, token_start=self.token_start, page_start=self.page_start,
            new_lens=self.new_lens, status=self.status, free_next_out=free_next_out)

        self.inv_freq = [rope_base ** (-2.0 * i / head_dim) for i in range(head_dim // 2)]
        self.freqs = binding.rope_freqs(self.inv_freq, device=device)
        self.block_tokens = max(n for n in range(1, binding.GEMV_MAX_BLOCK_TOKENS + 1) if page_size % n == 0)
        self.kind = {"bf16": binding.GEMV_CACHE_BF16, "fp8": binding.GEMV_CACHE_FP8,
                     "fp8_block": binding.GEMV_CACHE_FP8_BLOCK}[cache]
        self.workspace = binding.attn_workspace(self.q_heads, self.kv_heads, head_dim, self.kind, device=device)
        self.layers = []
        for l in range(spec["layers"]):
            self.layers.append(self._layer(l, seed, g))
        self._graph = None

    def _layer(self, l: int, seed: int, g) -> dict:
        H, Q, KV = self.spec["hidden"], self.spec["q_rows"], self.spec["kv_rows"]
        B, D, dev = self.batch, self.head_dim, self.device
        base = 16 * l
        d = dict(x=inputs.activations(B, H, seed=seed, index=base + 14, device=dev),
                 W=[inputs.weight(n, H, self.ldw_h, seed=seed, index=base + j, device=dev)
                    for j, n in enumerate((Q, KV, KV))],
                 Wo=inputs.weight(H, Q, self.ldw_q, seed=seed, index=base + 3, device=dev),
                 y=[torch.empty((B, n), dtype=torch.float32, device=dev) for n in (Q, KV, KV)],
                 q=torch.empty((B, Q), dtype=torch.bfloat16, device=dev),
                 out=torch.empty((B, Q), dtype=torch.bfloat16, device=dev),
                 o=torch.empty((B, H), dtype=torch.float32, device=dev))
        shape = (self.num_pages, self.page_size, self.kv_heads, D)
        scales, per_page = [None, None], self.page_size // self.block_tokens
        for i, n in enumerate(("k", "v")):
            d[n] = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
            if self.cache != "bf16":
                d[n] = (d[n] * 32).to(torch.float8_e4m3fn)
                scales[i] = torch.full((self.kv_heads,) if self.cache == "fp8" else
                                       (self.num_pages, per_page, self.kv_heads), 1.0 / 32, device=dev)
        d["scales"] = scales
        if self.cache == "fp8_block":
            scaled = dict(k_block_scale=scales[0], v_block_scale=scales[1], block_tokens=self.block_tokens,
                          scale_page_stride=per_page * self.kv_heads, scale_block_stride=self.kv_heads,
                          scale_head_stride=1)
        else:
            scaled = dict(k_scale=scales[0], v_scale=scales[1])
        d["cache"] = binding.kv_cache(
            d["k"], d["v"], num_pages=self.num_pages, page_size=self.page_size, kv_heads=self.kv_heads, head_dim=D,
            page_stride=self.page_size * KV, head_stride=D, slot_stride=KV,
            kind=self.kind, **scaled)
        d["rope"] = binding.rope_args(
            q=d["y"][0], k=d["y"][1], v=d["y"][2], q_out=d["q"], positions=self.positions, freqs=self.freqs,
            tokens=B, q_heads=self.q_heads, kv_heads=self.kv_heads, head_dim=D, rot_dim=D, q_stride=Q, k_stride=KV,
            v_stride=KV, q_out_stride=Q, slots=self.slots, rows=binding.GEMV_ROWS_F32)
        d["attn"] = binding.attn_args(
            q=d["q"], out=d["out"], lens=self.new_lens, requests=B, q_heads=self.q_heads, q_stride=Q, out_stride=Q,
            table=self.table, table_width=self.width, table_stride=self.width, scale=D ** -0.5,
            workspace=self.workspace, token_start=self.token_start, status=self.status, rows=B)
        d["segments"] = [(W, y, W.shape[0], self.ldw_h) for W, y in zip(d["W"], d["y"])]
        return d

    @property
    def launches(self) -> int:
        return 1 + 4 * len(self.layers)

    def run(self, stream=None) -> None:
        """One step, launch by launch."""
        H, Q, B = self.spec["hidden"], self.spec["q_rows"], self.batch
        binding.gemv_block_tables(self.tables, stream)
        for d in self.layers:
            binding.gemv_bf16_multi(d["segments"], d["x"], H, B, stream)
            binding.gemv_rope_append(d["rope"], d["cache"], stream)
            binding.gemv_attn_decode(d["attn"], d["cache"], stream)
            binding.gemv_bf16(d["Wo"], d["out"], d["o"], H, Q, B, self.ldw_q, stream)

    def capture(self) -> None:
        """The step as one CUDA graph. Nothing executes, but a first call on the
        device must have been made."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            self.run()
        self._graph = graph

    def launch(self) -> None:
        """Replay the captured step on the current stream."""
        self._graph.replay()

    def algorithmic_bytes(self) -> int:
        """Per step: weights, activations and projections' outputs as in
        DecodeStep; q, k and v rows read, q and the new slots written; the
        visible tokens' K and V and q read, the attention's output written."""
        H, Q, KV, B = self.spec["hidden"], self.spec["q_rows"], self.spec["kv_rows"], self.batch
        es = 2 if self.cache == "bf16" else 1
        scales = 0
        if self.cache == "fp8_block":    # those of the visible tokens read, of the new tokens' blocks read and written
            scales = 8 * self.kv_heads * (sum(-(-(n + 1) // self.block_tokens) for n in self.context) + 2 * B)
        layer = (roofline.algorithmic_bytes(Q + 2 * KV, H, B) + roofline.algorithmic_bytes(H, Q, B)
                 + B * (4 * (Q + 2 * KV) + 2 * Q + 2 * KV * es)
                 + 2 * sum(n + 1 for n in self.context) * KV * es + B * 4 * Q + scales)
        return len(self.layers) * layer
