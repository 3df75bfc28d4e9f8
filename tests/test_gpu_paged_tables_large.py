"""Page tables that many CTAs resize, against a list in Python; resizes and appends captured."""
import random
import threading

import pytest
import torch

from lossless_invariant_bit_gb300.paged import PagedCache
from tests.gpu_util import DEV
from tests.test_gpu_paged_tables import Model, cache_of, call, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_seqs,max_pages,n_pages,P", [
    (300, 40, 3000, 16), (2, 4000, 6000, 8), (1500, 3, 2500, 32), (17, 600, 7000, 256),
])
def test_growing_shrinking_and_refused_calls(n_seqs, max_pages, n_pages, P):
    """More than 4096 entries: two kernels, or one of many CTAs where nothing grows."""
    r = random.Random(n_seqs)
    t, m = cache_of(n_pages, P).tables(n_seqs, max_pages), Model(n_seqs, max_pages, n_pages, P)
    most = max_pages * P
    mean = n_pages * P // n_seqs
    kinds = {"grown": 0, "shrunk": 0, "refused": 0}
    for i in range(18):
        target = []
        for n in m.lens:
            x = r.random()
            if i % 3 == 1:  # a call that only shrinks
                target.append(n if x < 0.4 else 0 if x < 0.6 else r.randint(0, n))
            else:
                target.append(n if x < 0.2 else min(most, n + r.randint(1, 3)) if x < 0.5
                              else min(most, r.randint(0, mean)))
        if i % 6 == 4:  # that grows all the same, in one place; that is too long
            s = r.randrange(n_seqs)
            target[s] = m.lens[s] + 1
        elif i % 6 == 5:
            target[r.randrange(n_seqs)] = most + 1
        rows = sum(max(0, b - a) for a, b in zip(m.lens, target))
        only = i % 3 == 1
        got = call(t, m, target, 0 if only else rows + r.choice((0, 1, 500)))
        kinds["refused" if got is None else "shrunk" if only else "grown"] += 1
    assert all(kinds.values()), kinds


def test_many_rows_in_a_graph():
    """Both kernels of a resize of more than 1024 rows, replayed, against eager calls."""
    S, cols, n_pages, P, step = 40, 200, 4000, 16, 61
    t, m = cache_of(n_pages, P).tables(S, cols), Model(S, cols, n_pages, P)
    target = torch.zeros(S, dtype=torch.int32, device=DEV)
    slots = torch.zeros(S * step, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.resize(target, S * step, step, slots=slots)
        t.resize(target)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            target.add_(step)
            batch, _ = t.resize(target, S * step, step, slots=slots)
        back = torch.cuda.CUDAGraph()
        with torch.cuda.graph(back, stream=side):
            target.sub_(2 * step)
            t.resize(target)
        lens = 0
        for i in range(12):
            if i % 4 == 3:
                back.replay()
                side.synchronize()
                lens -= 2 * step
                assert m.resize([lens] * S, 0) is not None
            else:
                g.replay()
                side.synchronize()
                lens += step
                want = m.resize([lens] * S, S * step)
                assert batch.q_starts.tolist() == want[0] and slots.tolist() == want[1]
            same(t, m)
    assert t.cache.status() == 0


@pytest.mark.parametrize("page_dtype", [None, torch.float8_e4m3fn])
def test_a_prompts_step_in_a_graph(page_dtype):
    """Tables, append with queries and attention of more than 1024 rows: replays and eager
    calls leave the same bits."""
    H, G, D, P, S, step = 2, 4, 64, 16, 30, 50
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    q, k, v = (torch.randn((S * step, h, D), generator=g, device=DEV).bfloat16()
               for h in (H * G, H, H))
    qw, kw = (1 + 0.1 * torch.randn((2, D), generator=g, device=DEV)).bfloat16()
    ang = torch.rand((400, D // 2), generator=g, device=DEV) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()

    def a_cache():
        c = PagedCache(H, D, P, 900, torch.bfloat16, page_dtype=page_dtype)
        held = [x for x in (c.k, c.v, c.k_scales, c.v_scales) if x is not None]
        for x in held:
            x.view(torch.uint8).zero_()
        return c, c.tables(S, 200), torch.zeros(S, dtype=torch.int32, device=DEV), held

    def one(c, t, target):
        target.add_(step)
        batch, slots = t.resize(target, S * step, step)
        qo = c.append(batch, k, v, q=q, q_norm=qw, k_norm=kw, cos_sin=cs)
        return qo, c.attention(batch, qo), slots

    eager, graphed = a_cache(), a_cache()
    c, t, target, _ = graphed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one(c, t, target)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = one(c, t, target)
        target.fill_(step)
        for i in range(6):
            want = one(*eager[:3])
            torch.cuda.synchronize()
            if i:
                graph.replay()
                side.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(outs, want))
            for a, b in zip(eager[3], graphed[3]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert eager[0].status() == 0 and c.status() == 0


def test_threads_on_the_same_tables():
    """Calls of two threads on one stream: whatever their order, each page is one sequence's
    or free."""
    S, cols, n_pages, P = 40, 200, 5000, 16
    t = cache_of(n_pages, P).tables(S, cols)
    g = torch.Generator()
    g.manual_seed(1)
    targets = [torch.randint(0, 1900, (20, S), generator=g).to(torch.int32).to(DEV)
               for _ in range(2)]
    torch.cuda.synchronize()
    most = S * cols * P

    def work(rows):
        for x in rows:
            t.resize(x, most, slots=slots)

    slots = torch.empty(most, dtype=torch.int64, device=DEV)
    ts = [threading.Thread(target=work, args=(x,)) for x in targets]
    for x in ts:
        x.start()
    for x in ts:
        x.join()
    torch.cuda.synchronize()
    assert t.cache.status() == 0
    lens = t.kv_lens.tolist()
    assert any(lens == x[-1].tolist() for x in targets)
    pages = t.free_pages[:int(t.n_free)].tolist()
    for row, n in zip(t.page_table.tolist(), lens):
        pages += row[:-(-n // P)]
    assert sorted(pages) == list(range(n_pages))
