"""gemv_block_tables against its definition, number by number."""
import random

import pytest
import torch

from memory_bound_decode_gb300 import binding
from tests.blocks_ref import block_tables

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, lens, new, page, width, room, spare, seed=0, taken=0, stride=None, free_next=None, in_place=False):
        rng = random.Random(seed)
        self.lens, self.new, self.page, self.width, self.room = lens, new, page, width, room
        R = self.R = len(lens)
        have = [min(width, -(-max(0, n) // page)) for n in lens]
        self.num_pages = max(1, sum(have) + spare)
        order = list(range(self.num_pages))
        rng.shuffle(order)
        self.stride = stride or width
        self.table = [[-5] * self.stride for _ in range(R)]
        at = 0
        for r in range(R):
            self.table[r][:have[r]] = order[at:at + have[r]]
            at += have[r]
        self.free = [0] * taken + order[at:]
        self.free_next = taken if free_next is None else free_next
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        out = lambda n: torch.full((n + 2,), -99, dtype=torch.int32, device="cuda")  # noqa: E731
        self.t = dict(lens=dev(lens), new_tokens=dev(new), table=dev(self.table),
                      free_pages=dev(self.free or [0]), free_next=dev([self.free_next]))
        self.guarded = dict(slots=out(room), positions=out(room), token_start=out(R + 1), page_start=out(R),
                            new_lens=out(R), status=out(R), free_next_out=out(1))
        o = {n: x[1:-1] for n, x in self.guarded.items()}
        if in_place:
            o["new_lens"], o["free_next_out"] = self.t["lens"], self.t["free_next"]
        self.o = o
        self.args = binding.block_tables_args(requests=R, page_size=page, num_pages=self.num_pages, table_width=width,
                                              table_stride=self.stride, free_cap=len(self.free), max_tokens=room,
                                              **self.t, **o)

    def check(self, lens=None, free_next=None):
        want = block_tables(self.lens if lens is None else lens, self.new, self.table, self.page, self.width,
                            self.num_pages, self.free, self.free_next if free_next is None else free_next, self.room)
        for n in ("slots", "positions", "token_start", "page_start", "new_lens", "status"):
            assert self.o[n].tolist() == want[n], n
        assert self.o["free_next_out"].tolist() == [want["free_next"]]
        assert self.t["table"].tolist() == want["table"]
        for n, x in self.guarded.items():
            assert int(x[0]) == -99 and int(x[-1]) == -99, n
        return want

    def run(self):
        binding.gemv_block_tables(self.args)
        torch.cuda.synchronize()


@pytest.mark.parametrize("R,hi,new_hi,page,room,spare", [
    (1, 0, 1, 16, 1, 1), (1, 5000, 1, 16, 4, 1), (64, 4096, 1, 16, 64, 128), (7, 20, 9, 1, 64, 70),
    (40, 300, 50, 7, 2000, 400), (1024, 40, 3, 4, 4096, 2000), (1025, 40, 3, 4, 4096, 2000), (3000, 10, 2, 16, 9000, 5000),
    (5000, 9, 3, 8, 12000, 9000), (300, 100, 200, 16, 40000, 3000), (300, 100, 200, 16, 25000, 3000),
    (300, 100, 200, 16, 40000, 900), (20, 100, 8192, 128, 100000, 900),
])
def test_tables(R, hi, new_hi, page, room, spare):
    rng = random.Random(R + hi)
    lens = [rng.randint(0, hi) for _ in range(R)]
    new = [rng.randint(0, new_hi) for _ in range(R)]
    width = -(-(hi + new_hi) // page)
    s = Step(lens, new, page, width, room, spare, seed=R, taken=3)
    s.run()
    s.check()


def test_refusals_leave_the_others():
    """Every reason at once: negative, too long, past the room, out of pages; requests without tokens are served."""
    lens = [5, -1, 60, 16, 0, 3, 30, 0, 8, -2]
    new = [1, 1, 5, 1, -3, 0, 20, 0, 40, 0]
    for spare in (0, 1, 2, 9):
        for room in (1, 2, 6, 28, 40, 100):
            s = Step(lens, new, 16, 4, room, spare, taken=1)
            s.run()
            s.check()


@pytest.mark.parametrize("first", [-4, 2, 5, 1000])
def test_free_list_bounds(first):
    """A place in the free list outside it gives no page."""
    s = Step([16, 3, 32], [1, 1, 0], 16, 4, 8, 5, free_next=first)
    s.run()
    s.check()


def test_empty_free_list():
    s = Step([3, 16], [1, 1], 16, 4, 8, 0)
    s.run()
    assert s.check()["status"] == [0, 1]


def test_bad_page_numbers_give_no_slot():
    s = Step([20, 5], [2, 2], 16, 4, 4, 4)
    s.table[0][1] = s.num_pages
    s.table[1][0] = -1
    s.t["table"].copy_(torch.tensor(s.table, dtype=torch.int32))
    s.run()
    assert s.check()["slots"] == [-1] * 4


def test_wide_rows_are_left():
    s = Step([10, 40], [8, 9], 8, 7, 32, 9, stride=11)
    s.run()
    s.check()


def test_counts_past_32_bits():
    """Token counts whose sum passes 2^31: numbers stop at 2^31 - 1, the requests are refused."""
    big = 2 ** 31 - 1
    s = Step([0, 4, 4], [big, big, 1], 16, 4, 20, 4)
    s.run()
    assert s.check()["status"] == [2, 2, 3]


def test_in_place_state_under_replay():
    """lens and free_next advance themselves: a captured call replayed is one step after the other."""
    for R, room in ((5, 64), (5, 9000)):
        s = Step([0, 3, 15, 31, 7], [1, 2, 1, 5, 0], 16, 8, room, 12, in_place=True)
        s.run()
        want = s.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            binding.gemv_block_tables(s.args)
        for _ in range(6):
            graph.replay()
            torch.cuda.synchronize()
            want = s.check(lens=want["new_lens"], free_next=want["free_next"])
