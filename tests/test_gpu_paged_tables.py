"""Page tables on the GPU (ibp_paged_resize) against a list in Python."""
import random

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp
from lossless_invariant_bit_gb300.paged import PagedCache
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


class Model:
    """What the formulas say, one page after another."""

    def __init__(self, n_seqs, max_pages, n_pages, P):
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.lens, self.P, self.cols, self.n_pages = [0] * n_seqs, P, max_pages, n_pages
        self.free = list(range(n_pages))[::-1]

    def resize(self, target, n_tokens):
        """q_starts and slots, or None where the call cannot be served."""
        P = self.P
        have = [-(-n // P) for n in self.lens]
        want = [-(-n // P) for n in target]
        gone = sum(max(0, h - w) for h, w in zip(have, want))
        come = sum(max(0, w - h) for h, w in zip(have, want))
        rows = sum(max(0, t - n) for t, n in zip(target, self.lens))
        if (min(target) < 0 or max(want) > self.cols or rows > n_tokens
                or come > len(self.free) + gone):
            return None
        for s in reversed(range(len(target))):
            for i in reversed(range(want[s], have[s])):
                self.free.append(self.table[s][i])
        starts, slots = [0], []
        for s in range(len(target)):
            for i in range(have[s], want[s]):
                self.table[s][i] = self.free.pop()
            for pos in range(self.lens[s], target[s]):
                slots.append(self.table[s][pos // P] * P + pos % P)
            starts.append(len(slots))
        self.lens = list(target)
        return starts, slots


def cache_of(n_pages, P):
    return PagedCache(1, 16, P, n_pages, torch.float16, page_dtype=torch.float8_e4m3fn)


def same(t, m):
    assert t.kv_lens.tolist() == m.lens
    assert int(t.n_free) == len(m.free)
    assert t.free_pages[:len(m.free)].tolist() == m.free
    rows = t.page_table.tolist()
    for s, n in enumerate(m.lens):
        k = -(-n // m.P)
        assert rows[s][:k] == m.table[s][:k], s
    assert t._state.tolist()[1] == 0


def call(t, m, target, n_tokens):
    d = torch.tensor(target, dtype=torch.int32, device=DEV)
    slots = torch.full((n_tokens,), -7, dtype=torch.int64, device=DEV) if n_tokens else None
    got = t.resize(d, n_tokens, slots=slots)
    want = m.resize(target, n_tokens)
    if want is None:
        assert t.cache.status() == ibp.IBP_ERANGE
        if got:
            assert got[0].q_starts.tolist() == [0] * (len(target) + 1)
            assert bool((slots == -7).all())
    else:
        assert t.cache.status() == 0
        if n_tokens:
            assert got[0].q_starts.tolist() == want[0]
            assert slots[:len(want[1])].tolist() == want[1]
            assert bool((slots[len(want[1]):] == -7).all())  # rows behind the last
        else:
            assert got is None
    same(t, m)
    return want


@pytest.mark.parametrize("n_seqs,max_pages,n_pages,P", [
    (1, 1, 1, 8), (3, 7, 20, 16), (20, 40, 300, 32), (257, 9, 900, 16), (700, 5, 2000, 8),
    (2, 300, 500, 256), (1, 3000, 3500, 16),
])
def test_random_lengths(n_seqs, max_pages, n_pages, P):
    r = random.Random(n_seqs)
    t, m = cache_of(n_pages, P).tables(n_seqs, max_pages), Model(n_seqs, max_pages, n_pages, P)
    same(t, m)
    served = 0
    for i in range(25):
        target = []
        for n in m.lens:
            x = r.random()
            if x < 0.3:
                target.append(n)
            elif x < 0.6:
                target.append(min(max_pages * P, n + r.randint(1, 3)))
            elif x < 0.75:
                target.append(0)
            else:
                target.append(r.randint(0, max(1, min(max_pages * P, 2 * n_pages * P // n_seqs))))
        rows = sum(max(0, b - a) for a, b in zip(m.lens, target))
        served += call(t, m, target, rows + r.choice((0, 0, 1, 300, -1 if rows > 1 else 0))) \
            is not None
    assert served


def test_a_growth_that_is_taken_back():
    t, m = cache_of(64, 16).tables(4, 16), Model(4, 16, 64, 16)
    call(t, m, [100, 16, 0, 33], 149)
    before = [x.clone() for x in (t.page_table, t.kv_lens, t.free_pages, t.n_free)]
    call(t, m, [117, 17, 90, 33], 120)
    call(t, m, [100, 16, 0, 33], 0)
    for a, b in zip(before[1:], (t.kv_lens, t.free_pages, t.n_free)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("target,n_tokens", [
    ([129, 0], 200),          # beyond the table
    ([-1, 0], 10),            # no length
    ([40, 41], 80),           # more tokens than rows
    ([40, 0], 0),             # growth in a call that only shrinks
    ([128, 97], 400),         # 8 + 7 pages of 14
])
def test_a_call_that_cannot_be_served_changes_nothing(target, n_tokens):
    t, m = cache_of(14, 16).tables(2, 8), Model(2, 8, 14, 16)
    assert call(t, m, target, n_tokens) is None
    assert call(t, m, [128, 96], 224) is not None  # and the next one is
    assert call(t, m, [127, 97], 1) is None  # its last page is needed still
    assert call(t, m, [112, 97], 1) is not None  # it is returned and taken


def test_state_that_cannot_be():
    """Lengths or a list's length that no call leaves: refused, nothing is read by them."""
    t = cache_of(14, 16).tables(2, 8)
    target = torch.tensor([5, 5], dtype=torch.int32, device=DEV)
    for bad in (-1, 15, 2 ** 31 - 1):
        t.n_free.fill_(bad)
        batch, _ = t.resize(target, 10)
        assert t.cache.status() == ibp.IBP_ERANGE and batch.q_starts.tolist() == [0, 0, 0]
        assert t.kv_lens.tolist() == [0, 0] and int(t.n_free) == bad
    t.n_free.fill_(14)
    for bad in (-1, 129, 2 ** 31 - 1):
        t.kv_lens.fill_(bad)
        t.resize(target, 10)
        assert t.cache.status() == ibp.IBP_ERANGE and t.kv_lens.tolist() == [bad, bad]


def test_calls_in_a_graph():
    t, m = cache_of(64, 16).tables(3, 16), Model(3, 16, 64, 16)
    target = torch.zeros(3, dtype=torch.int32, device=DEV)
    slots = torch.zeros(12, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        target.add_(0)
        t.resize(target, 12, 4, slots=slots)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            target.add_(4)
            batch, _ = t.resize(target, 12, 4, slots=slots)
        for i in range(1, 9):
            g.replay()
            side.synchronize()
            want = m.resize([4 * i] * 3, 12)
            assert batch.q_starts.tolist() == want[0] and slots.tolist() == want[1]
            same(t, m)
    assert t.cache.status() == 0


def test_a_16_bit_cache_has_tables_too():
    c = PagedCache(2, 64, 16, 8, torch.float16)
    t = c.tables(1, 8)
    batch, slots = t.resize(torch.tensor([20], dtype=torch.int32, device=DEV), 20)
    k = torch.randn((20, 2, 64), device=DEV).half()
    c.append(batch, k, k)
    assert torch.equal(c.key_rows()[slots].view(torch.float16).view(20, 2, 64), k)
    out = c.attention(batch, k)
    assert c.status() == 0 and torch.equal(out[0], k[0])
