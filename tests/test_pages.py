"""Page tables, slots and positions of a step against a plain form that takes a request at a time: exact."""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import step as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def state(rng, lens, page, cols, spare, capacity=None):
    """(table, lens, free, n_free): every request's pages lie anywhere, `spare` are free."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    pool = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n]
        at += n
    free = np.full(pages if capacity is None else capacity, -7, np.int32)
    free[:spare] = pool[at:][:len(free)]
    return table, np.array(lens, np.int32), free, min(spare, len(free))


class Both:
    """The same state on the GPU and in the plain form; a step has to leave both alike."""

    def __init__(self, table, lens, free, n_free, page, wide=0):
        self.plain = [table.copy(), lens.copy(), free.copy(), n_free]
        # rows may lie further apart than they are long
        base = torch.full((len(lens), table.shape[1] + wide), -9, dtype=torch.int32, device="cuda")
        base[:, :table.shape[1]] = gpu(table)
        self.base, self.page = base, page
        self.gpu = [base[:, :table.shape[1]], gpu(lens), gpu(free), gpu([n_free])]

    def step(self, change, total=None):
        change = np.asarray(change, np.int32)
        if total is None:
            total = int(np.maximum(change, 0).sum())
        got = fm.pages_update(self.gpu[0], self.gpu[1], gpu(change), self.gpu[2], self.gpu[3], self.page, total)
        t, n, free, n_free = self.plain
        self.plain[3], *want = plain.pages(t, n, change, free, n_free, self.page, total)
        for name, a, b in zip(got._fields, got, want):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert self.gpu[3].item() == self.plain[3]
        for name, a, b in zip(("table", "lens", "free"), self.gpu, self.plain):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert (self.base[:, t.shape[1]:] == -9).all()
        return got


@pytest.mark.parametrize("B,page,cols", [(1, 64, 8), (3, 1, 40), (31, 16, 20), (33, 48, 9), (256, 64, 12), (1025, 100, 3),
                                         (4095, 7, 6), (8192, 32, 4)])
def test_steps(B, page, cols):
    rng = np.random.default_rng(B)
    room = cols * page
    lens = rng.integers(0, room + 1, B)
    lens[rng.random(B) < 0.2] = 0
    both = Both(*state(rng, lens, page, cols, 3 * B), page, wide=B % 5)
    for kind in range(5):
        n = both.plain[1].astype(np.int64)
        change = {0: np.ones(B, np.int64),                                            # a decode step
                  1: np.where(rng.random(B) < 0.3, -n, rng.integers(0, 5, B)),        # some end
                  2: -rng.integers(0, 4, B),                                          # drafted tokens are not accepted
                  3: rng.integers(-room, room, B),                                    # anything
                  4: np.where(n == 0, rng.integers(0, room + 1, B), 1)}[kind]         # prompts and decode steps
        both.step(change, None if kind % 2 else int(np.maximum(change, 0).sum()) + 3)


def test_the_stack_runs_out_in_order():
    rng = np.random.default_rng(1)
    lens = [64, 10, 63, 64, 0, 128, 5]
    both = Both(*state(rng, lens, 64, 4, 3), 64)
    # 64 -> 2 pages more, 10 -> none, 63 -> none, 64 -> 2 (the stack has 1), 0 -> 1 (not any more), 128 -> 1, 5 -> none
    got = both.step([65, 1, 1, 66, 1, 1, 59])
    assert got.changed.tolist() == [65, 1, 1, 0, 0, 0, 59]
    assert both.plain[3] == 1
    # what shrinks makes room in the same step, and is what is taken first
    got = both.step([-65, 1, 0, 64, 1, -1, 0])
    assert got.changed.tolist() == [-65, 1, 0, 64, 1, -1, 0]


def test_rows_that_are_full_and_odd_arguments():
    rng = np.random.default_rng(2)
    both = Both(*state(rng, [128, 127, 0, 1], 32, 4, 9), 32)
    assert both.step([1, 2, 129, 2 ** 31 - 1], total=300).changed.tolist() == [0, 0, 0, 0]
    assert both.step([-2 ** 31, -2 ** 31, -1, 0]).changed.tolist() == [-128, -127, 0, 0]
    # lengths outside the table's room, a count past the stack's end or below nothing: taken as the nearest that is there
    for n_free in (-5, 10 ** 6):
        both = Both(np.arange(12, dtype=np.int32).reshape(3, 4), np.array([-3, 1000, 7], np.int32),
                    np.arange(20, 26, dtype=np.int32), n_free, 8)
        both.step([3, 0, 2])
    # pages that are not there have no slots
    both = Both(np.array([[3, -1, 5]], np.int32), np.array([3], np.int32), np.array([9], np.int32), 0, 2)
    assert both.step([1]).slots.tolist() == [-1]
    # more pages come back than the stack holds: the last ones are dropped
    both = Both(*state(rng, [100, 200, 60], 16, 16, 2, capacity=9), 16)
    both.step([-100, -150, 3])
    assert both.plain[3] == 9


def test_empty_calls():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fm.pages_update(none.view(0, 4), none, none, none, one, 64, 0)
    assert got.starts.tolist() == [0] and got.changed.numel() == 0
    got = fm.pages_update(none.view(0, 4), none, none, none, one, 64, 5)
    assert got.slots.tolist() == [-1] * 5
    both = Both(np.empty((2, 0), np.int32), np.zeros(2, np.int32), np.arange(3, dtype=np.int32), 3, 64)
    assert both.step([1, 0]).changed.tolist() == [0, 0]
    # fewer rows than tokens: the lengths grow all the same
    both = Both(*state(np.random.default_rng(3), [5, 6], 4, 9, 9), 4)
    both.step([7, 9], total=3)


def test_many_tokens_in_a_few_requests():
    rng = np.random.default_rng(4)
    both = Both(*state(rng, [0, 70001, 3, 0], 64, 3000, 2200), 64)
    both.step([60001, 1, 0, 65537])
    both.step([-60001, -70002, 9999, 1])


def test_captured_and_replayed():
    # a decode step of static buffers, lengths and the stack carried from replay to replay
    rng = np.random.default_rng(5)
    both = Both(*state(rng, [3, 0, 17, 64], 4, 40, 60), 4)
    change = gpu([1, 1, 1, 1])
    fm.pages_update(*both.gpu[:2], gpu([0] * 4), *both.gpu[2:], 4, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fm.pages_update(*both.gpu[:2], change, *both.gpu[2:], 4, 6)
    for i in range(9):
        new = np.array([1, 1, 1, 1]) if i < 6 else rng.integers(-9, 2, 4)
        change.copy_(gpu(new))
        graph.replay()
        t, n, free, n_free = both.plain
        both.plain[3], *want = plain.pages(t, n, new, free, n_free, 4, 6)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
        assert both.gpu[3].item() == both.plain[3] and np.array_equal(both.gpu[0].cpu().numpy(), t)
        assert np.array_equal(both.gpu[1].cpu().numpy(), n) and np.array_equal(both.gpu[2].cpu().numpy(), free)


def test_a_large_step_captured_and_replayed():
    # many CTAs for the tokens, and the lengths by a kernel of their own
    rng = np.random.default_rng(7)
    both = Both(*state(rng, [0, 100, 31], 32, 900, 2500), 32)
    change = gpu([0, 0, 0])
    fm.pages_update(*both.gpu[:2], change, *both.gpu[2:], 32, 20000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fm.pages_update(*both.gpu[:2], change, *both.gpu[2:], 32, 20000)
    for new in ([9000, 7000, 1], [1, 1, 1], [-9001, 3000, -33], [20000, 20000, 30000], [0, 0, 0]):
        change.copy_(gpu(new))
        graph.replay()
        t, n, free, n_free = both.plain
        both.plain[3], *want = plain.pages(t, n, new, free, n_free, 32, 20000)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
        assert both.gpu[3].item() == both.plain[3] and np.array_equal(both.gpu[0].cpu().numpy(), t)
        assert np.array_equal(both.gpu[1].cpu().numpy(), n) and np.array_equal(both.gpu[2].cpu().numpy(), free)


def test_on_another_stream():
    rng = np.random.default_rng(6)
    both = Both(*state(rng, [100] * 40, 16, 30, 300), 16)
    side = torch.cuda.Stream()
    change = gpu([33] * 40)
    torch.cuda.synchronize()
    got = fm.pages_update(*both.gpu[:2], change, *both.gpu[2:], 16, 33 * 40, stream=side)
    side.synchronize()
    t, n, free, n_free = both.plain
    _, *want = plain.pages(t, n, np.full(40, 33), free, n_free, 16, 33 * 40)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
