"""gemv_block_tables where token numbers reach the end of 31 bits, and in place with more requests than a CTA sums."""
import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests.blocks_ref import block_tables

pytestmark = pytest.mark.gpu

MAX32 = 2 ** 31 - 1


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_tokens_past_the_last_number_are_refused():
    """A refused request's tokens keep their numbers; one whose own come behind 2^31 - 1 finds no room."""
    lens, new = [0, 3, 5], [MAX32, 5, 0]
    out = dict(slots=torch.full((MAX32,), -5, dtype=torch.int32, device="cuda"),
               positions=torch.full((MAX32,), -5, dtype=torch.int32, device="cuda"))
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 0] = 7, 6
    free = i32([1, 2, 3])
    small = {n: torch.full((k,), -5, dtype=torch.int32, device="cuda")
             for n, k in (("token_start", 4), ("page_start", 3), ("new_lens", 3), ("status", 3), ("free_next_out", 1))}
    lens_t, new_t, next_t = i32(lens), i32(new), i32([0])
    args = binding.block_tables_args(lens=lens_t, new_tokens=new_t, requests=3, page_size=16, num_pages=8,
                                     table=table, table_width=4, table_stride=4, free_pages=free, free_cap=3,
                                     free_next=next_t, max_tokens=MAX32, **out, **small)
    binding.gemv_block_tables(args)
    torch.cuda.synchronize()
    assert small["status"].tolist() == [2, 3, 0]
    assert small["token_start"].tolist() == [0, MAX32, MAX32, MAX32]
    assert small["page_start"].tolist() == [-1, -1, 0] and small["new_lens"].tolist() == [0, 3, 5]
    assert small["free_next_out"].tolist() == [0] and table.tolist() == [[-1] * 4, [7, -1, -1, -1], [6, -1, -1, -1]]
    assert int(out["slots"].max()) == -1 and int(out["slots"].min()) == -1
    assert int(out["positions"].max()) == 0 and int(out["positions"].min()) == 0


@pytest.mark.parametrize("requests", [1023, 1024, 1025, 5000])
@pytest.mark.parametrize("top", [1, 3, 40])
def test_state_advanced_in_place(requests, top):
    """lens and free_next moved on by the call itself, three times over, with requests refused on the way."""
    page, width, num_pages = 16, 6, 4096
    lens = [(i * 7) % 60 for i in range(requests)]
    held = sum(-(-n // page) for n in lens)
    num_pages += held
    order = torch.randperm(num_pages, generator=torch.Generator().manual_seed(requests)).tolist()
    table, at = [], 0
    for n in lens:
        k = -(-n // page)
        table.append(order[at:at + k] + [-1] * (width - k))
        at += k
    free = order[at:at + requests]                 # runs out for the larger counts
    new = [(i * 5) % (top + 1) for i in range(requests)]
    room = sum(new) - top                          # the last ones with new tokens find no room
    state = dict(lens=i32(lens), free_next=i32([2]), table=i32(table), new=i32(new), free=i32(free))
    out = {n: torch.empty(k, dtype=torch.int32, device="cuda")
           for n, k in (("slots", room), ("positions", room), ("token_start", requests + 1), ("page_start", requests),
                        ("status", requests))}
    args = binding.block_tables_args(
        lens=state["lens"], new_tokens=state["new"], requests=requests, page_size=page, num_pages=num_pages,
        table=state["table"], table_width=width, table_stride=width, free_pages=state["free"], free_cap=len(free),
        free_next=state["free_next"], max_tokens=room, new_lens=state["lens"], free_next_out=state["free_next"], **out)
    next_page = 2
    for _ in range(3):
        want = block_tables(lens, new, table, page, width, num_pages, free, next_page, room)
        for t in out.values():
            t.fill_(-9)
        binding.gemv_block_tables(args)
        torch.cuda.synchronize()
        for n, t in out.items():
            assert t.tolist() == want[n], n
        assert state["lens"].tolist() == want["new_lens"] and state["table"].tolist() == want["table"]
        assert state["free_next"].tolist() == [want["free_next"]]
        lens, next_page = want["new_lens"], want["free_next"]
