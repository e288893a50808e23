"""Pages and places of a step's tokens against their definition, one row at a time: whole numbers, equal."""
import itertools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def KV():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from model_free_suffix_gb300 import build
    build.build()
    from model_free_suffix_gb300 import KVCache
    return KVCache


class Server:
    """The definition: tables and the free list as lists."""

    def __init__(self, pages, P, B, width):
        self.P, self.width, self.pages = P, width, pages
        self.table, self.held = [[-1] * width for _ in range(B)], [0] * B
        self.free, self.count = list(range(pages - 1, -1, -1)), pages

    def assign(self, keep, new, N):
        B, P, errors = len(keep), self.P, set()
        got, bad = list(new), [False] * B
        for b in range(B):
            if keep[b] < 0 or new[b] < 0 or keep[b] > self.held[b] * P or keep[b] + new[b] > self.width * P:
                got[b], bad[b] = 0, True
                errors.add("length")
        at = 0
        for b in range(B):
            at += got[b]
            if at > N and got[b] > 0:
                got[b] = 0
                errors.add("room")
        need = [self.held[b] if bad[b] else -(-(keep[b] + got[b]) // P) for b in range(B)]
        for b in range(B):
            for j in range(need[b], self.held[b]):
                self.free[self.count] = self.table[b][j]
                self.table[b][j] = -1
                self.count += 1
        have, wanted = self.count, 0
        for b in range(B):
            want = need[b] - self.held[b]
            if want > 0:
                wanted += want
                if wanted > have:
                    got[b] = 0
                    errors.add("room")
                    continue
                for j in range(self.held[b], need[b]):
                    self.count -= 1
                    self.table[b][j] = self.free[self.count]
            self.held[b] = need[b]
        lens = [0 if bad[b] else keep[b] + got[b] for b in range(B)]
        rows, positions, slots = [-1] * N, [0] * N, [-1] * N
        i = 0
        for b in range(B):
            for p in range(keep[b], keep[b] + got[b]):
                rows[i], positions[i], slots[i] = b, p, self.table[b][p // P] * P + p % P
                i += 1
        return lens, [0] + list(itertools.accumulate(got)), positions, slots, rows, errors


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Pair:
    def __init__(self, KV, pages, P, B, width):
        self.kv = KV(num_pages=pages, page_size=P, kv_heads=1, head_dim=64, max_batch=B, max_pages_per_row=width)
        self.pages, self.ref = self.kv.new_pages(), Server(pages, P, B, width)

    def step(self, keep, new, N):
        from model_free_suffix_gb300 import _lib as L
        plan = self.kv.assign(self.pages, _i32(keep), _i32(new), N)
        lens, starts, positions, slots, rows, errors = self.ref.assign(keep, new, N)
        assert plan.seq_lens.tolist() == lens and plan.q_start.tolist() == starts
        assert plan.positions.tolist() == positions and plan.rows.tolist() == rows and plan.slots.tolist() == slots
        want = (L.KV_ERR_LENGTH if "length" in errors else 0) | (L.KV_ERR_ROOM if "room" in errors else 0)
        assert self.kv.get_error(clear=True) == want
        self.check()
        return plan

    def check(self):
        B = len(self.ref.held)
        assert np.array_equal(self.pages.block_table.cpu().numpy()[:B], np.array(self.ref.table))
        assert self.pages.held.tolist()[:B] == self.ref.held and self.pages.free_count.tolist() == [self.ref.count]
        assert self.pages.free.tolist() == self.ref.free


@pytest.mark.parametrize("B,P", [(1, 16), (3, 32), (33, 64), (257, 16), (1025, 128), (2100, 16)])
def test_steps(KV, B, P):
    """Rows that come with prompts, decode, reject and finish; some steps without tokens."""
    rng = np.random.default_rng(B)
    width = 24
    p = Pair(KV, B * 12 + 8, P, B, width)
    have = np.zeros(B, np.int64)
    for step in range(8):
        keep = np.maximum(0, have - rng.integers(0, 2 * P, B) * (rng.random(B) < 0.4))
        new = rng.integers(0, 18, B)
        over = rng.random(B) < 0.2
        keep[over], new[over] = 0, 0
        coming = (keep == 0) & (rng.random(B) < 0.5)
        new[coming] = rng.integers(0, 6 * P, int(coming.sum()))
        if step == 5:
            keep[:], new[:] = 0, 0
        new = np.minimum(new, width * P - keep)
        plan = p.step(keep.tolist(), new.tolist(), max(1, int(new.sum()) + int(rng.integers(0, 3))))
        have = plan.seq_lens.cpu().numpy().astype(np.int64)


def test_rows_behind_the_call_keep_their_pages(KV):
    p = Pair(KV, 40, 16, 5, 8)
    p.step([0] * 5, [20, 33, 1, 64, 16], 200)
    before = p.pages.block_table[3:].clone()
    plan = p.kv.assign(p.pages, _i32([20, 0, 1]), _i32([13, 0, 40]), 100)
    assert plan.seq_lens.tolist() == [33, 0, 41] and torch.equal(p.pages.block_table[3:], before)
    assert p.pages.held.tolist() == [3, 0, 3, 4, 1]


def test_too_few_pages(KV):
    """A row that does not fit gets nothing; those behind it that need no page still get theirs."""
    p = Pair(KV, 10, 16, 6, 10)
    p.step([0] * 6, [40, 20, 0, 70, 3, 1], 300)       # 3 + 2 + 0 + 5 pages: the last two find none
    p.step([40, 20, 0, 70, 0, 0], [8, 13, 0, 10, 5, 0], 300)
    p.step([48, 1, 0, 0, 0, 0], [1, 1, 16, 17, 16, 80], 300)  # pages given back in the same call are handed out


def test_too_little_room_for_tokens(KV):
    p = Pair(KV, 60, 16, 6, 10)
    p.step([0] * 6, [40, 20, 0, 70, 3, 1], 100)
    p.step([40, 20, 0, 0, 0, 0], [1, 1, 0, 1, 1, 1], 2)
    p.step([41, 21, 0, 0, 0, 0], [1, 1, 1, 1, 1, 1], 0)


def test_lengths_that_make_no_sense(KV):
    p = Pair(KV, 60, 16, 6, 10)
    p.step([0] * 6, [40, 20, 10, 70, 3, 1], 200)
    p.step([-1, 33, 10, 70, 4, 1], [1, 1, -1, 91, 0, 2 ** 31 - 1], 200)
    p.step([2 ** 31 - 1, 20, 10, 70, 3, 1], [2 ** 31 - 1, 1, 1, 90, -2 ** 31, 1], 200)
    p.step([48, 32, 16, 80, 16, 16], [1, 1, 1, 1, 1, 1], 200)


def test_damaged_state_is_reported(KV):
    """Nothing is written out of place whatever the state holds."""
    from model_free_suffix_gb300 import _lib as L
    kv = KV(num_pages=20, page_size=16, kv_heads=1, head_dim=64, max_batch=3, max_pages_per_row=6)
    pages = kv.new_pages()
    kv.assign(pages, _i32([0, 0, 0]), _i32([40, 50, 60]), 200)
    assert kv.get_error() == 0
    guard = pages.free_count.clone()
    for count in (-7, 2 ** 31 - 1):
        pages.free_count.fill_(count)
        kv.assign(pages, _i32([40, 50, 60]), _i32([20, 20, 20]), 60)
        assert kv.get_error(clear=True) & L.KV_ERR_PAGE
    pages = kv.new_pages()
    pages.held.copy_(_i32([7, -1, 2]))
    plan = kv.assign(pages, _i32([40, 0, 20]), _i32([1, 1, 1]), 60)
    assert kv.get_error(clear=True) & L.KV_ERR_LENGTH
    assert plan.seq_lens.tolist() == [0, 0, 21]
    # more pages given back than there are: the list stays within its end
    pages = kv.new_pages()
    pages.held.copy_(_i32([6, 6, 6]))
    kv.assign(pages, _i32([0, 0, 0]), _i32([0, 0, 0]), 4)
    assert kv.get_error(clear=True) & L.KV_ERR_PAGE
    assert pages.free_count.tolist() == [20] and guard.numel() == 1
    # ids that are no pages are not turned into slots
    pages = kv.new_pages()
    pages.free.fill_(10 ** 6)
    plan = kv.assign(pages, _i32([0, 0, 0]), _i32([3, 0, 0]), 4)
    assert kv.get_error(clear=True) & L.KV_ERR_PAGE and plan.slots.tolist() == [-1] * 4


@pytest.mark.parametrize("held", [-1, -2, -7, -2 ** 31])
def test_a_row_that_holds_less_than_nothing(KV, held):
    """It is passed over: its row of the table, those beside it and what lies around the table stay as they were."""
    from model_free_suffix_gb300 import _lib as L
    B, width, around = 5, 6, 4
    kv = KV(num_pages=40, page_size=16, kv_heads=1, head_dim=64, max_batch=B, max_pages_per_row=width)
    pages = kv.new_pages()
    tables = torch.full((around + B + around, width), -77, dtype=torch.int32, device="cuda")
    lists = torch.full((40 + 40 + 40,), -55, dtype=torch.int32, device="cuda")
    tables[around:around + B], lists[40:80] = pages.block_table, pages.free
    pages.block_table, pages.free = tables[around:around + B], lists[40:80]
    kv.assign(pages, _i32([0] * B), _i32([40, 50, 33, 1, 16]), 200)
    assert kv.get_error() == 0
    before, free, count = tables.clone(), lists.clone(), pages.free_count.item()
    for row in (0, 2, 4):
        for keep, new in ((0, 0), (0, 90), (16, 1)):
            at = pages.held.clone()
            at[row] = held
            pages.held.copy_(at)
            keeps, news = [40, 50, 33, 1, 16], [0] * B
            keeps[row], news[row] = keep, new
            plan = kv.assign(pages, _i32(keeps), _i32(news), 100)
            assert kv.get_error(clear=True) == L.KV_ERR_LENGTH
            keeps[row] = 0
            assert plan.seq_lens.tolist() == keeps and plan.q_start.tolist() == [0] * (B + 1)
            assert torch.equal(tables, before) and torch.equal(lists, free) and pages.free_count.item() == count
            assert pages.held.tolist() == at.tolist()
            pages.held.copy_(_i32([3, 4, 3, 1, 1]))


def test_rows_that_claim_more_pages_than_32_bits_count(KV):
    """8192 rows of 2^18 pages each, of a cache of 1000: the list takes the first and no others."""
    from model_free_suffix_gb300 import _lib as L
    B, width, N = 8192, (1 << 18) + 7, 1000
    kv = KV(num_pages=N, page_size=16, kv_heads=1, head_dim=64, max_batch=B, max_pages_per_row=width)
    pages = kv.new_pages()
    pages.block_table.fill_(3)
    pages.block_table[0, :N] = torch.arange(N, dtype=torch.int32, device="cuda")
    lists = torch.full((3 * N,), -55, dtype=torch.int32, device="cuda")
    pages.free = lists[N:2 * N]
    pages.held.fill_(width)
    pages.free_count.zero_()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    plan = kv.assign(pages, zero, zero, 1)
    assert kv.get_error(clear=True) == L.KV_ERR_PAGE
    assert pages.free.tolist() == list(range(N)) and pages.free_count.tolist() == [N]
    assert bool((lists[:N] == -55).all()) and bool((lists[2 * N:] == -55).all())
    assert not bool(pages.held.any()) and bool((pages.block_table == -1).all()) and plan.q_start[-1].item() == 0
    kv.close()


def test_outputs_that_are_left_out_and_lengths_in_place(KV):
    p = Pair(KV, 40, 16, 4, 8)
    from model_free_suffix_gb300 import PagePlan
    keep, new = _i32([0, 0, 0, 0]), _i32([5, 40, 0, 17])
    plan = PagePlan(keep, torch.empty(5, dtype=torch.int32, device="cuda"))
    p.kv.assign(p.pages, keep, new, total=100, out=plan)           # seq_lens takes keep's place
    assert keep.tolist() == [5, 40, 0, 17] and plan.q_start.tolist() == [0, 5, 45, 45, 62]
    p.kv.assign(p.pages, keep, new, total=100, out=PagePlan(new, plan.q_start, slots=torch.empty(100, dtype=torch.int32, device="cuda")))
    assert new.tolist() == [10, 80, 0, 34]
    assert p.kv.get_error() == 0


def test_no_rows(KV):
    p = Pair(KV, 4, 16, 2, 2)
    plan = p.kv.assign(p.pages, _i32([]), _i32([]), 3)
    assert plan.q_start.tolist() == [0] and plan.slots.tolist() == [-1] * 3 and plan.positions.tolist() == [0] * 3


def test_many_tokens(KV):
    """Prompts of thousands of tokens: the tokens are the work."""
    p = Pair(KV, 1000, 64, 9, 400)
    p.step([0] * 9, [20000, 1, 0, 9000, 4097, 0, 3, 12000, 511], 46000)
    p.step([20000, 1, 0, 0, 4097, 0, 3, 12000, 511], [1, 1, 1, 25000, 0, 0, 1, 1, 1], 25010)


def test_captured(KV):
    """One graph, replayed over many steps."""
    kv = KV(num_pages=64, page_size=16, kv_heads=1, head_dim=64, max_batch=4, max_pages_per_row=16)
    pages, ref = kv.new_pages(), Server(64, 16, 4, 16)
    keep, new, plan = _i32([0] * 4), _i32([0] * 4), kv.new_plan(4, 120)
    kv.assign(pages, keep, new, out=plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.assign(pages, keep, new, out=plan)
    for a, c in (([0] * 4, [30, 1, 17, 64]), ([30, 1, 17, 60], [5, 5, 5, 5]), ([35, 0, 20, 65], [16, 0, 1, 100]), ([0] * 4, [0] * 4)):
        keep.copy_(_i32(a))
        new.copy_(_i32(c))
        graph.replay()
        lens, starts, positions, slots, rows, _ = ref.assign(a, c, 120)
        assert plan.seq_lens.tolist() == lens and plan.q_start.tolist() == starts and plan.slots.tolist() == slots
        assert plan.positions.tolist() == positions and plan.rows.tolist() == rows
        assert pages.free.tolist() == ref.free and pages.free_count.tolist() == [ref.count]
    assert kv.get_error() == 0
