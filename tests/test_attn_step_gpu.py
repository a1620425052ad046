"""The attention operators as a decode step uses them: block tables, the QKV
projection, rotary positions with the cache write, attention and the output
projection, chained, captured and replayed. Each stage is held to 64 bits on
the actual outputs of the stage before it."""
import pytest
import torch

from memory_bound_decode_gb300 import binding, workloads
from tests import attn_util as au

pytestmark = pytest.mark.gpu

TINY = dict(layers=2, hidden=512, intermediate=512, vocab=64, q_rows=512, kv_rows=256)


def check(step, lens):
    """One step that has run, with `lens` tokens a request before it."""
    B, D, P = step.batch, step.head_dim, step.page_size
    assert step.status.tolist() == [0] * B and step.positions.tolist() == lens
    assert step.token_start.tolist() == list(range(B + 1))
    table = step.table.cpu()
    for r, n in enumerate(lens):
        assert int(step.slots[r]) == int(table[r, n // P]) * P + n % P
    assert step.new_lens.tolist() == [n + 1 for n in lens]
    used = [int(g) for r, n in enumerate(lens) for g in table[r, :n // P + 1]]
    assert len(set(used)) == len(used), "two requests share a page"
    inv = torch.tensor(step.inv_freq, dtype=torch.float64)
    slots = step.slots.cpu().long()
    for d in step.layers:
        H, Q = step.spec["hidden"], step.spec["q_rows"]
        x = d["x"].double().cpu()
        for W, y in zip(d["W"], d["y"]):
            w = W[:, :H].double().cpu()
            assert ((y.double().cpu() - x @ w.T).abs() <= 1e-5 * (x.abs() @ w.abs().T)).all()
        pos = step.positions[None]
        zero = torch.zeros(D // 2, dtype=torch.int32)
        rows = [y.view(B, -1, D) for y in d["y"]]
        q, size = au.turn(rows[0], pos, inv, zero, D, False)
        tol = au.BF16 * q.abs() + 1.01 * 2.0 ** -20 * size + 1e-38
        assert ((d["q"].view(B, -1, D).double().cpu() - q).abs() <= tol).all()
        k, size = au.turn(rows[1], pos, inv, zero, D, False)
        values = []
        for n, want, sz in (("k", k, size), ("v", rows[2].double().cpu(), torch.zeros_like(size))):
            pool = d[n].view(torch.uint8).cpu().view(d[n].dtype).double().reshape(-1, step.kv_heads, D)
            if step.cache == "fp8":
                pool = pool / 32
                tol = (au.E4M3 * want.abs()).clamp(min=2.0 ** -15) + 1.01 * 2.0 ** -20 * sz
            else:
                tol = au.BF16 * want.abs() + 1.01 * 2.0 ** -20 * sz + 1e-38
            assert ((pool[slots] - want).abs() <= tol).all(), n
            values.append(pool)
        for r, n in enumerate(lens):
            at = torch.tensor([int(table[r, j // P]) * P + j % P for j in range(n + 1)])
            out, z, mass, sz = au.attend(d["q"][r].cpu().view(-1, D), values[0][at], values[1][at], D ** -0.5)
            tol, _ = au.attn_bounds(out, z, mass, sz, n + 1, D, step.cache)
            assert ((d["out"][r].double().cpu().view(-1, D) - out).abs() <= tol).all(), r
        a, w = d["out"].double().cpu(), d["Wo"][:, :Q].double().cpu()
        assert ((d["o"].double().cpu() - a @ w.T).abs() <= 1e-5 * (a.abs() @ w.abs().T)).all()
    assert binding.gemv_device_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("context,page", [([0, 15, 16, 300, 1], 16), ([7], 24), ([100] * 16, 7)])
def test_chained_step(cache, context, page):
    step = workloads.AttentionStep(TINY, context, batch=len(context), cache=cache, page_size=page)
    step.run()
    torch.cuda.synchronize()
    check(step, context)


def test_replayed_steps_append_one_token_after_the_other():
    lens = [0, 14, 31, 200]
    step = workloads.AttentionStep(TINY, lens, batch=4, page_size=16, advance=True, room=24)
    step.run()
    torch.cuda.synchronize()
    check(step, lens)
    step.capture()
    for i in range(1, 21):
        for j, d in enumerate(step.layers):
            d["x"].copy_(au.randn(100 * i + j, *d["x"].shape, dtype=torch.bfloat16))
        step.launch()
        torch.cuda.synchronize()
        if i in (1, 2, 3, 17, 20):
            check(step, [n + i for n in lens])


def test_step_without_room_leaves_its_request_alone():
    """The table's row is full: the request is refused, its slot skipped, the others go on."""
    lens = [31, 5]
    step = workloads.AttentionStep(TINY, lens, batch=2, page_size=16, advance=True, room=1)   # rows of two pages
    for _ in range(2):
        step.run()
    torch.cuda.synchronize()
    before = [d["k"].clone() for d in step.layers]
    step.run()
    torch.cuda.synchronize()
    assert step.status.tolist() == [2, 0] and step.lens.tolist() == [32, 8]
    assert int(step.slots[0]) == -1
    for d, k in zip(step.layers, before):
        changed = (d["k"] != k).flatten(2).any(-1)
        assert changed.nonzero().tolist() == [[int(step.slots[1]) // 16, int(step.slots[1]) % 16]]


def test_refuses_bad_arguments():
    for bad in (dict(context=[1, 2], batch=3), dict(context=-1), dict(context=4, cache="int8"),
                dict(context=4, head_dim=96), dict(context=4, batch=17)):
        with pytest.raises(ValueError):
            workloads.AttentionStep(TINY, **bad)
