"""Block tables and slot maps built on the GPU, against a plan made request by request."""
import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu


class State:
    """A pool and the tables of B requests, on the GPU and as arrays."""

    def __init__(self, seed, B, page, width, spare, held=None):
        self.g = np.random.default_rng(seed)
        self.page = page
        self.held = (self.g.integers(0, width + 1, B) if held is None else np.asarray(held)).astype(np.int32)
        n = int(self.held.sum())
        self.pages = n + spare + 3
        ids = self.g.permutation(self.pages).astype(np.int32)
        self.table = np.full((B, width), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :self.held[b]] = ids[at:at + self.held[b]]
            at += self.held[b]
        self.free = np.concatenate([ids[at:at + spare], np.full(n + 3, -7, np.int32)])
        self.count = spare
        import speculative_decoding_verification_15_gb300 as pkg

        self.pkg = pkg
        self.pool = pkg.PagePool(self.cuda(self.free), self.cuda([self.count]))
        self.dtable, self.dheld = self.cuda(self.table), self.cuda(self.held)

    @staticmethod
    def cuda(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def lengths(self, new):
        """What each request keeps of what it holds, and up to `new` more tokens."""
        keep = (self.g.random(len(self.held)) * (self.held * self.page + 1)).astype(np.int32)
        return keep, self.g.integers(0, new + 1, len(keep)).astype(np.int32)

    def call(self, keep, new, n_out):
        return self.pkg.kv_plan(self.pool, self.dtable, self.dheld, self.cuda(keep), self.cuda(new), self.page, n_out)

    def check(self, got, keep, new, n_out):
        want = U.plan(self.free, self.count, self.table, self.held, keep, new, self.page, n_out)
        for name in ("cu_new", "seq_len", "slot", "position", "status"):
            np.testing.assert_array_equal(got[name].cpu().numpy(), want[name], err_msg=name)
        np.testing.assert_array_equal(self.dtable.cpu().numpy(), want["table"])
        np.testing.assert_array_equal(self.dheld.cpu().numpy(), want["held"])
        self.count = len(want["free"])
        assert int(self.pool.count) == self.count
        self.free = self.pool.free.cpu().numpy()
        np.testing.assert_array_equal(self.free[:self.count], want["free"])
        self.table, self.held = want["table"], want["held"].astype(np.int32)
        return want


@pytest.mark.parametrize("B,page,width,new", [(1, 16, 3, 1), (7, 64, 5, 200), (64, 64, 20, 8), (256, 32, 9, 9),
                                              (257, 16, 30, 40), (1500, 128, 4, 60), (8192, 16, 6, 20)])
@pytest.mark.parametrize("scarce", [False, True])
def test_rounds(B, page, width, new, scarce):
    """Several calls one after another: requests grow, shrink and end, pages wander."""
    s = State(B + scarce, B, page, width, B // 8 if scarce else B * (new // page + 2))
    seen = set()
    for i in range(4):
        keep, fresh = s.lengths(new)
        if i == 2:  # a third of them end
            keep[::3] = fresh[::3] = 0
        n_out = int(fresh.sum()) + (0, 5, 300, 1)[i]
        seen |= set(s.check(s.call(keep, fresh, n_out), keep, fresh, n_out)["status"].tolist())
    assert 0 in seen


@pytest.mark.parametrize("B", [5, 200, 5000])
@pytest.mark.parametrize("spare", [0, 1, 3])
def test_a_pool_that_runs_out(B, spare):
    """Requests that only grow: those before the list's end are served, and those that lack
    nothing; given pages serve takers of the same call."""
    s = State(B + spare, B, 16, 40, spare * B // 4)
    keep = (s.held * 16 - s.g.integers(0, 8, B) * (s.held > 0)).astype(np.int32)
    new = np.minimum(s.g.integers(0, 50, B), 40 * 16 - keep).astype(np.int32)
    keep[1], new[1] = 0, 0
    want = s.check(s.call(keep, new, int(new.sum())), keep, new, int(new.sum()))
    assert 0 in want["status"]
    assert B == 5 or 7 in want["status"]  # of five, one that ends may serve the others


@pytest.mark.parametrize("B", [9, 900])
def test_bad_lengths(B):
    s = State(5, B, 32, 6, 4 * B)
    keep, new = s.lengths(70)
    keep[1], new[2], new[4] = -1, -3, 6 * 32 + 1
    keep[5] = s.held[5] * 32 + 1
    s.held[6] = s.held[8] = 0
    s.table[[6, 8]] = -1
    keep[[6, 8]] = 0
    s.dtable.copy_(s.cuda(s.table))
    bad = s.held.copy()
    bad[6], bad[8] = 7, -1
    s.dheld.copy_(s.cuda(bad))
    s.held = bad
    n_out = int(np.maximum(new, 0).sum()) - int(max(new[-1], 0)) - 1  # the last request's rows do not fit
    new[-1] = max(new[-1], 1)
    want = s.check(s.call(keep, new, n_out), keep, new, n_out)
    assert (want["status"][[1, 2, 4, 5, 6, 8, -1]] == 2).all()


def test_nothing_to_plan():
    s = State(1, 0, 16, 4, 5)
    none = np.zeros(0, np.int32)
    s.check(s.call(none, none, 3), none, none, 3)
    s = State(2, 4, 16, 4, 5)
    zero = np.zeros(4, np.int32)
    s.check(s.call(zero, zero, 0), zero, zero, 0)  # everybody ends


def test_tables_without_pages():
    s = State(3, 5, 16, 0, 5, held=np.zeros(5))
    keep, new = np.zeros(5, np.int32), np.array([0, 1, 0, 2, 0], np.int32)
    assert s.check(s.call(keep, new, 3), keep, new, 3)["status"].tolist() == [0, 2, 0, 2, 0]


@pytest.mark.parametrize("B", [50, 3000])
def test_taking_and_giving_back_restores_the_pool(B):
    s = State(B, B, 16, 12, 9 * B)
    keep = (s.held * 16).astype(np.int32)
    new = np.minimum(s.g.integers(0, 100, B), 12 * 16 - keep).astype(np.int32)
    free, table = s.free[:s.count].copy(), s.table.copy()
    s.check(s.call(keep, new, int(new.sum())), keep, new, int(new.sum()))
    zero = np.zeros(B, np.int32)
    s.check(s.call(keep, zero, 0), keep, zero, 0)
    np.testing.assert_array_equal(s.free[:s.count], free)
    np.testing.assert_array_equal(s.table, table)


def test_many_rows_and_one_long_request():
    s = State(11, 3, 128, 900, 900, held=[0, 5, 0])
    keep, new = np.array([0, 600, 0], np.int32), np.array([110001, 1, 0], np.int32)
    s.check(s.call(keep, new, 110100), keep, new, 110100)
    s.check(s.call(new * 0, new * 0, 70), new * 0, new * 0, 70)


def test_captured_rounds():
    """A captured call takes each replay's lengths, and goes on from the pool it finds."""
    s = State(21, 40, 16, 9, 400)
    keep, new = s.lengths(20)
    dk, dn = s.cuda(keep), s.cuda(new)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = s.pkg.kv_plan(s.pool, s.dtable, s.dheld, dk, dn, s.page, 900)
    for _ in range(3):
        dk.copy_(s.cuda(keep))
        dn.copy_(s.cuda(new))
        graph.replay()
        s.check(got, keep, new, 900)
        keep, new = s.lengths(20)


def test_many_pages_of_few_requests():
    """A few requests with long tables end and start: their pages move without new tokens."""
    s = State(23, 40, 16, 1200, 100)
    zero = np.zeros(40, np.int32)
    s.check(s.call(zero, zero, 3), zero, zero, 3)
    new = s.g.integers(0, 1200 * 16 + 1, 40).astype(np.int32)
    new[np.cumsum(-(-new // 16)) > s.count] = 1
    s.check(s.call(zero, new, 2000), zero, new, 2000)  # most tokens' rows do not fit: those requests fail
    s.check(s.call(zero, new, int(new.sum())), zero, new, int(new.sum()))


def test_another_stream():
    s = State(22, 300, 32, 9, 3000)
    keep, new = s.lengths(20)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = s.pkg.kv_plan(s.pool, s.dtable, s.dheld, s.cuda(keep).long(), s.cuda(new).long(), s.page, 7000, stream=stream)
    torch.cuda.synchronize()
    s.check(got, keep, new, 7000)
