"""kv_pages_advance against the rule written out in Python, step after step, and the conservation of pages."""

import random

import pytest
import torch

from paged_util import i32

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


class Plain:
    """The rule, one entry at a time."""

    def __init__(self, table, lengths, page, n_pages, free):
        self.table, self.len, self.page, self.n = [list(r) for r in table], list(lengths), page, n_pages
        self.free, self.missing = list(free), 0

    def used(self, n):
        return min(-(-n // self.page), len(self.table[0]))

    def advance(self, rows, n_rows):
        room = self.n - len(self.free)
        back, pos, slots, start = [], [], [], [0]
        for i, r in enumerate(rows):
            old = max(self.len[i], 0)
            now = min(max(old + r, 0), MOST)
            for e in range(self.used(old), self.used(now)):
                if self.free:
                    self.table[i][e] = self.free.pop(0)
                else:
                    self.table[i][e] = -1
                    self.missing += 1
            for e in range(self.used(now), self.used(old)):
                if 0 <= self.table[i][e] < self.n and len(back) < room:
                    back.append(self.table[i][e])
                self.table[i][e] = -1
            self.len[i] = now
            start.append(start[-1] + max(r, 0))
        self.free += back
        for i, r in enumerate(rows):
            for p in range(self.len[i] - max(r, 0), self.len[i]):
                pos.append(p)
                page = self.table[i][p // self.page] if 0 <= p and p // self.page < len(self.table[0]) else -1
                slots.append(page * self.page + p % self.page if 0 <= page < self.n else -1)
        fit = lambda v: (v + [-1] * n_rows)[:n_rows]
        return start, fit(pos), fit(slots)


def ring_of(free):
    ring, (head, count, missing) = free.ring.tolist(), free.state.tolist()
    return [ring[(head + k) % len(ring)] for k in range(count)], missing


def verify(kvc, pages, free, plain, rows, n_rows):
    got = kvc.kv_pages_advance(pages, free, i32(rows), n_rows)
    want = plain.advance(rows, n_rows)
    for g, w, what in zip(got, want, ("row_start", "positions", "slots")):
        assert g.tolist() == w, what
    assert pages.lengths.tolist() == plain.len
    assert pages.table.tolist() == plain.table
    assert ring_of(free) == (plain.free, plain.missing)


def fresh(kvc, n_seq, width, page, n_pages, order=None):
    table = torch.full((n_seq, width), -1, dtype=torch.int32, device="cuda")
    pages = kvc.PageTable(table, torch.zeros(n_seq, dtype=torch.int32, device="cuda"), page)
    free = kvc.FreePages(n_pages, order)
    return pages, free, Plain(table.tolist(), [0] * n_seq, page, n_pages, order or range(n_pages))


@pytest.mark.parametrize("n_seq,width,page,n_pages,longest", [
    (1, 3, 16, 3, 60), (5, 8, 16, 25, 100), (64, 40, 16, 900, 500), (33, 5, 48, 40, 300), (300, 12, 32, 700, 400),
    (1024, 6, 16, 2500, 90), (1025, 6, 16, 2500, 90), (2500, 3, 64, 3000, 150)])
def test_steps_of_a_scheduler(kvc, n_seq, width, page, n_pages, longest):
    # prompts, tokens, rewinds and ends; pages run out now and then, and lengths pass the table
    rng = random.Random(n_seq)
    order = list(range(n_pages))
    rng.shuffle(order)
    pages, free, plain = fresh(kvc, n_seq, width, page, n_pages, order)
    for step in range(12):
        rows = []
        for i in range(n_seq):
            n = plain.len[i]
            u = rng.random()
            if n == 0:
                rows.append(rng.randint(1, longest) if u < 0.5 else 0)
            elif u < 0.2:
                rows.append(-n if u < 0.15 else -2 ** 31)
            elif u < 0.3:
                rows.append(-rng.randint(1, n))
            else:
                rows.append(1 if u < 0.9 else rng.randint(0, longest))
        total = sum(max(r, 0) for r in rows)
        verify(kvc, pages, free, plain, rows, max(0, total + rng.choice([0, 0, 5, -3])))
        held = [p for r in pages.table.tolist() for p in r if p >= 0]
        ring, _ = ring_of(free)
        assert sorted(held + ring) == list(range(n_pages))
    verify(kvc, pages, free, plain, [-2 ** 31] * n_seq, 0)
    assert free.free()[0] == n_pages


def test_many_rows(kvc):
    # more rows than the one CTA places, in few and in many sequences
    for n_seq, each in ((2, 30000), (1500, 9)):
        pages, free, plain = fresh(kvc, n_seq, 30000 // 16 + 1 if n_seq == 2 else 2, 16, 4000)
        verify(kvc, pages, free, plain, [each] * n_seq, each * n_seq + 7)
        verify(kvc, pages, free, plain, [-each + 1] * n_seq, 3)


def test_pages_that_run_out(kvc):
    pages, free, plain = fresh(kvc, 3, 10, 16, 4)
    verify(kvc, pages, free, plain, [33, 30, 20], 83)    # 3 + 2 + 2 pages of 4
    assert free.free() == (0, 3)
    verify(kvc, pages, free, plain, [1, 1, -20], 2)      # its holes give nothing back
    verify(kvc, pages, free, plain, [-40, 1, 0], 1)
    verify(kvc, pages, free, plain, [0, 0, 16], 16)      # what came back is there now


def test_what_is_given_back_is_taken_by_the_next_call(kvc):
    pages, free, plain = fresh(kvc, 2, 2, 16, 2)
    verify(kvc, pages, free, plain, [32, 0], 32)
    verify(kvc, pages, free, plain, [-32, 16], 16)       # not by this one
    assert pages.table.tolist()[1] == [-1, -1] and free.free() == (2, 1)
    verify(kvc, pages, free, plain, [0, 16], 16)
    assert pages.table.tolist()[1] == [-1, 0]


def test_lengths_at_their_limits(kvc):
    pages, free, plain = fresh(kvc, 4, 3, 16, 20)
    pages.lengths.copy_(i32([MOST - 1, -5, 0, 40]))
    plain.len[:] = [MOST - 1, -5, 0, 40]
    pages.table.copy_(i32([[0, 1, 2], [-1, -1, -1], [-1, -1, -1], [7, -1, 1 << 30]]))
    plain.table = pages.table.tolist()
    free = kvc.FreePages(20, [3, 4, 5, 6])
    plain.free = [3, 4, 5, 6]
    verify(kvc, pages, free, plain, [100, 2, -2 ** 31, -2 ** 31], 0)
    assert pages.lengths.tolist() == [MOST, 2, 0, 0]
    verify(kvc, pages, free, plain, [-MOST, 0, 0, 0], 0)


def test_any_state_is_safe(kvc):
    for state in ([-7, 5, 0], [3, 1 << 30, -4], [1 << 30, -9, 2 ** 31 - 1]):
        pages, free, _ = fresh(kvc, 2, 3, 16, 5)
        free.state.copy_(i32(state))
        start, pos, slots = kvc.kv_pages_advance(pages, free, i32([20, 30]), 50)
        assert start.tolist() == [0, 20, 50] and pos.tolist() == list(range(20)) + list(range(30))
        assert all(-1 <= s < 80 for s in slots.tolist())
        head, count, missing = free.state.tolist()
        assert 0 <= head < 5 and 0 <= count <= 5 and missing >= 0


def test_given_outputs_and_none_of_them(kvc):
    pages, free, plain = fresh(kvc, 3, 4, 16, 20)
    rs, pos, slots = i32([9] * 4), i32([9] * 6), i32([9] * 6)
    out = kvc.kv_pages_advance(pages, free, i32([1, 2, 0]), 5, rs, pos[:5], slots[:5])
    assert out[0] is rs and rs.tolist() == [0, 1, 3, 3]
    assert pos.tolist() == [0, 0, 1, -1, -1, 9] and slots[5] == 9
    st = kvc.lib.kv_pages_advance(pages.addr, free.addr, i32([1, 0, 0]).data_ptr(), rs.data_ptr(), 1, None, None,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0 and pages.lengths.tolist() == [2, 2, 0]


def test_no_sequences(kvc):
    nobody = kvc.PageTable(torch.empty(0, 1, dtype=torch.int32, device="cuda"), i32([]), 16)
    start, pos, slots = kvc.kv_pages_advance(nobody, kvc.FreePages(3), i32([]), 2)
    assert start.tolist() == [0] and pos.tolist() == [-1, -1] and slots.tolist() == [-1, -1]


def test_replayed_graph_goes_on(kvc):
    # a decode loop: each replay takes the sequences one token further
    pages, free, plain = fresh(kvc, 5, 6, 16, 25)
    verify(kvc, pages, free, plain, [3, 15, 16, 0, 40], 74)
    ones = i32([1, 1, 1, 0, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = kvc.kv_pages_advance(pages, free, ones, 4)
    torch.cuda.synchronize()
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        want = plain.advance([1, 1, 1, 0, 1], 4)
        assert [t.tolist() for t in out] == [list(w) for w in want]
        assert pages.table.tolist() == plain.table and ring_of(free) == (plain.free, plain.missing)
