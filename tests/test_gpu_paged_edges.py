"""The paged K/V cache at its edges, against plain 64-bit implementations with the
bounds of test_gpu_paged.py."""
import math
import threading

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp, paged
from tests.gpu_util import DEV
from tests.test_gpu_paged import F64, U, Setup, near, rope_table, turn

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    """Calls of several threads share their stream's workspace; tiles here are cut, so
    their pieces go through it, in batches of one kernel, of the other, and of both."""
    sets = [Setup([300, 1, 1, 5], [3001, 4000, 77, 2000], G=8, D=128, dtype=torch.bfloat16, seed=1),
            Setup([1, 1], [9001, 3], G=4, H=3, D=64, seed=2),
            Setup([700, 1], [5000, 4999], G=7, D=128, dtype=torch.bfloat16, seed=3)]
    want = [st.cache.attention(st.batch, st.q, lse=True) for st in sets]
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(len(sets))

    def calls(i):
        st = sets[i]
        begin.wait()
        got = [st.cache.attention(st.batch, st.q, lse=True) for _ in range(150)]
        torch.cuda.current_stream().synchronize()
        wrong.extend(i for a in got if not (torch.equal(a[0], want[i][0])
                                            and torch.equal(a[1], want[i][1])))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert all(st.cache.status() == 0 for st in sets)


def test_stream_handle_zero_is_the_default_stream():
    assert paged._as_stream(0).cuda_stream == 0
    side = torch.cuda.Stream()
    assert paged._as_stream(side.cuda_stream).cuda_stream == side.cuda_stream
    assert paged._as_stream(side) is side
    st = Setup([1, 9], [40, 30], G=2, D=64)
    want = st.cache.attention(st.batch, st.q)
    assert torch.equal(st.cache.attention(st.batch, st.q, stream=0), want)


def test_empty_arguments_are_not_absent_ones():
    """A tensor without elements has a null pointer, which tells the library that it
    was not given: attention over no pages is not attention over every key."""
    st = Setup([2], [40], G=2, D=64, poison=False)
    k = torch.zeros((2, 2, 64), dtype=st.dtype, device=DEV)
    with pytest.raises(ValueError):
        st.cache.attention(st.batch, st.q, pages=torch.zeros((2, 2, 0), dtype=torch.int32,
                                                             device=DEV))
    for shape in ((0, 64), (64, 0)):
        with pytest.raises(ValueError):
            st.cache.append(st.batch, k, k, q=st.q, cos_sin=torch.zeros(shape, device=DEV))
    with pytest.raises(ValueError):
        st.cache.append(st.batch, k, k, q=st.q[:, :0])


# 4 new tokens at positions 30 to 33 of pages of 16: the last page begins with the third of
# them.  4 x 4 rows of a K/V head go to the step kernel, 4 x 16 to the chunk kernel.
@pytest.mark.parametrize("G", [1, 4, 16, 40])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_a_bad_page_zeroes_only_rows_that_see_it(G, bad):
    for window, page, need in ((0, 2, [2, 3]), (0, 0, [0, 1, 2, 3]), (16, 0, [0]),
                               (18, 0, [0, 1, 2]), (15, 0, [])):
        st = Setup([4, 1], [34, 50], G=G, D=64, P=16, seed=G)
        want, lse0 = st.cache.attention(st.batch, st.q, lse=True, window=window)
        st.table[0, page] = bad
        out, lse = st.cache.attention(st.batch, st.q, lse=True, window=window)
        assert st.cache.status() == (ibp.IBP_ERANGE if need else ibp.IBP_OK)
        for t in range(5):
            if t in need:
                assert not bool(out[t].any()) and bool((lse[t] == -math.inf).all()), (window, t)
            else:
                assert torch.equal(out[t], want[t]) and torch.equal(lse[t], lse0[t]), (window, t)


@pytest.mark.parametrize("G,n,bad", [(4, 4, 1), (4, 4, 1249), (8, 30, 1), (8, 30, 1249)])
def test_a_bad_page_of_a_cut_tile_zeroes_only_rows_that_see_it(G, n, bad):
    """The sequence's blocks are cut over all CTAs: pieces that saw the page and pieces
    that did not are joined.  Pages from `bad` on are out of range."""
    L = 20002
    st = Setup([n], [L], G=G, H=1, D=128, P=16, dtype=torch.bfloat16, seed=G)
    want, lse0 = st.cache.attention(st.batch, st.q, lse=True)
    first = (L - n) // 16 + 1 if bad > 1 else 1  # the first page that begins among new tokens
    see = torch.arange(L - n, L, device=DEV) >= first * 16
    assert bool(see.any())
    st.table[0, first:] = -1
    out, lse = st.cache.attention(st.batch, st.q, lse=True)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert not bool(out[see].any()) and bool((lse[see] == -math.inf).all())
    assert torch.equal(out[~see], want[~see]) and torch.equal(lse[~see], lse0[~see])


def test_a_bad_page_of_a_list_zeroes_its_token():
    st = Setup([3, 1], [60, 50], G=20, D=64, P=16, seed=2)
    pages = torch.tensor([[0, 2], [1, 3], [0, 1], [0, 3]], dtype=torch.int32, device=DEV)
    pages = pages[:, None].expand(4, 2, 2).contiguous()
    want = st.cache.attention(st.batch, st.q, pages=pages)
    st.table[0, 3] = -1
    out = st.cache.attention(st.batch, st.q, pages=pages)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert not bool(out[1].any())
    assert all(torch.equal(out[t], want[t]) for t in (0, 2, 3))


def test_append_and_bounds_with_tokens_before_the_first_position():
    """More new tokens than the sequence has positions: the tokens at positions 0 on
    are appended (attention, scores and selection serve them), the others refused."""
    q_lens, kv_lens, G, D, P = [5, 3, 2, 20], [2, 0, 40, 19], 2, 64, 8
    st = Setup(q_lens, kv_lens, G=G, D=D, P=P, seed=1, poison=False)
    H, T = st.H, st.T
    k = torch.randn((T, H, D), generator=st.g, device=DEV).to(st.dtype)
    v = torch.randn((T, H, D), generator=st.g, device=DEV).to(st.dtype)
    cs = rope_table(64, D)
    kb, vb = st.k.clone(), st.v.clone()
    q = st.cache.append(st.batch, k, v, q=st.q, cos_sin=cs)
    assert st.cache.status() == ibp.IBP_ERANGE
    wrote = torch.zeros((st.n_pages, P), dtype=torch.bool, device=DEV)
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        lo, before = st.starts[s], max(0, n - L)
        assert not bool(q[lo:lo + before].any())
        pos = torch.arange(L - n + before, L, device=DEV)
        rows = slice(lo + before, lo + n)
        page, slot = st.table[s, pos // P].long(), pos % P
        wrote[page, slot] = True
        near(q[rows], *turn(st.q[rows], None, cs[pos], D, False), st.dtype, D)
        near(st.k[page, slot], *turn(k[rows], None, cs[pos], D, False), st.dtype, D)
        assert torch.equal(st.v[page, slot], v[rows])
    assert torch.equal(st.k[~wrote], kb[~wrote]) and torch.equal(st.v[~wrote], vb[~wrote])
    bounds = torch.full((st.n_pages, H, 2, D), 7.0, dtype=st.dtype, device=DEV)
    ref = bounds.clone()
    st.cache.update_bounds(st.batch, bounds)
    assert st.cache.status() == ibp.IBP_OK
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        for p in range(max(0, L - n) // P, -(-L // P)):
            kk = st.k[st.table[s, p].long()][:min(P, L - p * P)]
            ref[st.table[s, p].long()] = torch.stack([kk.amin(0), kk.amax(0)], 1)
    assert torch.equal(bounds, ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,G,H,lists", [(1, 4, 160, False), (3, 4, 160, False),
                                         (4, 4, 160, True), (40, 4, 1, False), (60, 1, 2, False)])
@pytest.mark.parametrize("gap", [8.0, 14.0, 15.5, 16.0])
def test_weights_far_below_the_largest(n, G, H, lists, gap, dtype):
    """Four keys with score `gap` and values of zero, 3000 others with score 0: the
    result is made of weights exp(-gap) alone (2^-23 at 16, below fp16's normal
    numbers).  A weight may round by u, or by the subnormals' 2^-25 after the kernels have
    lifted the largest to 2^11 at least."""
    L, D, seqs = 3000, 64, 4 if H > 2 else 1
    st = Setup([n] * seqs, [L] * seqs, G=G, H=H, D=D, P=16, dtype=dtype, seed=7)
    st.q.zero_()
    st.q[:, :, 5] = 4.0  # gap / 4 is exact
    for s in range(seqs):
        st.K[s].zero_()
        st.K[s][:128:32, :, 5] = gap / 4
        st.V[s] = (512 + 512 * torch.rand((L, H, D), generator=st.g, device=DEV)).to(dtype)
        st.V[s][:128:32] = 0
        st.put(s)
    pages = None
    if lists:
        pages = torch.arange(st.cols, dtype=torch.int32, device=DEV)
        pages = pages.expand(st.T, H, -1).contiguous()
    out, lse = st.cache.attention(st.batch, st.q, scale=1.0, pages=pages, lse=True)
    u, e = U[dtype], 2.0 ** -24
    d = 2 * (2 * D * e * gap + 2.0 ** -20 * gap + 2.0 ** -20)
    for s in range(seqs):
        v = st.V[s].to(F64)
        for t in range(n):
            p = torch.full((L - n + t + 1,), math.exp(-gap), dtype=F64, device=DEV)
            p[:128:32] = 1
            ref = torch.einsum("k,khd->hd", p / p.sum(), v[:len(p)]).repeat_interleave(G, 0)
            bound = u * ref + (u + 2 * d + 2.0 ** -20) * ref
            if dtype == torch.float16:
                bound = bound + len(p) * 2.0 ** -36 * v.max() + 2.0 ** -25
            row = st.starts[s] + t
            diff = (out[row].to(F64) - ref).abs()
            assert bool((diff <= bound).all()), (s, t, (diff / ref).max().item())
            total = gap + math.log(float(p.sum()))
            assert float((lse[row].to(F64) - total).abs().max()) <= d / 2 + 2.0 ** -22 * total + \
                2.0 ** -20


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (24, 80)])
def test_scores_of_pages_with_infinite_keys(G, D, dtype):
    """sum_d max(q lo, q hi) as it is written: an infinite bound that the other one
    outdoes has no part in it; 0 * inf is NaN."""
    P, L, n = 8, 700, 5
    st = Setup([n], [L], G=G, D=D, P=P, dtype=dtype, seed=G)
    K = st.K[0]
    K[3, 0, 7] = math.inf
    K[20, 1, 3] = -math.inf
    K[40:48, 0, 9] = -math.inf  # both bounds of a channel
    K[60, 0, 2], K[61, 0, 2] = math.inf, -math.inf
    K[100, 0, 11] = math.inf
    K[300, 1, 4], K[301, 1, 6] = math.inf, -math.inf
    st.q[:, :, 11] = 0
    bounds = torch.zeros((st.n_pages, st.H, 2, D), dtype=dtype, device=DEV)
    for p in range(-(-L // P)):
        kk = K[p * P:(p + 1) * P]
        bounds[st.table[0, p]] = torch.stack([kk.amin(0), kk.amax(0)], 1)
    got = st.cache.page_scores(st.batch, st.q, bounds).to(F64)
    assert st.cache.status() == ibp.IBP_OK
    b = bounds[st.table[0].long()].to(F64)
    lo, hi = b[:, None, :, None, 0], b[:, None, :, None, 1]  # [pages, 1, H, 1, D]
    q = st.q.view(1, n, st.H, G, D).to(F64)
    term = torch.maximum(q * lo, q * hi)
    want = term.sum(-1).amax(-1).permute(1, 2, 0)
    big = q.abs() * torch.maximum(lo.abs(), hi.abs())
    big = torch.where(torch.isfinite(big), big, torch.where(torch.isfinite(term), term.abs(), 0.0))
    tol = (4 * D * 2.0 ** -24 * big.sum(-1).amax(-1)).permute(1, 2, 0)
    for t in range(n):
        vis = (L - n + t) // P + 1
        g, w = got[t, :, :vis], want[t, :, :vis]
        assert torch.equal(torch.isnan(g), torch.isnan(w))
        assert torch.equal(torch.isinf(g), torch.isinf(w))
        fin = torch.isfinite(w)
        assert torch.equal(g[~fin & ~torch.isnan(w)], w[~fin & ~torch.isnan(w)])
        assert bool(((g - w).abs() <= tol[t, :, :vis])[fin].all())


def test_the_bindings_functions_make_the_same_calls():
    """ibp.ibp_paged_*: one function to each C entry point, which PagedCache passes by."""
    st = Setup([3, 40], [70, 300], G=4, D=64, poison=False)
    c, b, ws = st.cache, st.batch, torch.empty(ibp.PAGED_WORKSPACE_BYTES, dtype=torch.uint8,
                                               device=DEV)
    H, D, T = st.H, st.D, st.T
    qkv = torch.randn((T, 6 * H, D), generator=st.g, device=DEV).to(st.dtype)
    q, k, v = qkv[:, :4 * H], qkv[:, 4 * H:5 * H], qkv[:, 5 * H:]
    w = (1 + 0.1 * torch.randn(D, generator=st.g, device=DEV)).to(st.dtype)
    cs = rope_table(300, D)
    row = 6 * H * D * 2
    want_q = c.append(b, k, v, q=q, q_norm=w, k_norm=w, cos_sin=cs, pairs=True)
    pages = [st.k.clone(), st.v.clone()]
    st.k.zero_(), st.v.zero_()
    for s in range(2):
        st.put(s)
    got_q = torch.empty_like(want_q)
    ibp.ibp_paged_append(c.handle, b.desc, k, v, row, q, row, got_q, 4 * H * D * 2, 4 * H, w, w,
                         1e-6, cs, 300, D, True)
    assert torch.equal(got_q, want_q)
    wrote = torch.zeros((st.n_pages, st.P), dtype=torch.bool, device=DEV)
    for s, (n, L) in enumerate(zip(st.q_lens, st.kv_lens)):
        pos = torch.arange(L - n, L, device=DEV)
        wrote[st.table[s, pos // st.P].long(), pos % st.P] = True
    assert torch.equal(st.k[wrote], pages[0][wrote]) and torch.equal(st.v[wrote], pages[1][wrote])
    want, want_lse = c.attention(b, got_q, window=50, lse=True)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    ibp.ibp_paged_attention(c.handle, b.desc, got_q, 4 * H * D * 2, 4 * H, out, lse, D ** -0.5,
                            True, 50, None, 0, ws, ibp.PAGED_WORKSPACE_BYTES)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    bounds = [torch.zeros((st.n_pages, H, 2, D), dtype=st.dtype, device=DEV) for _ in range(2)]
    c.update_bounds(b, bounds[0])
    ibp.ibp_paged_bounds(c.handle, b.desc, bounds[1])
    assert torch.equal(*bounds)
    want = c.page_scores(b, got_q, bounds[0])
    scores = torch.empty_like(want)
    ibp.ibp_paged_scores(c.handle, b.desc, got_q, 4 * H * D * 2, 4 * H, bounds[0], scores)
    assert torch.equal(scores, want)
    picked = c.select_pages(b, scores, 5)
    got = torch.empty_like(picked)
    ibp.ibp_paged_select(c.handle, b.desc, scores, 5, got)
    assert torch.equal(got, picked)
    want = c.attention(b, got_q, pages=picked)
    ibp.ibp_paged_attention(c.handle, b.desc, got_q, 4 * H * D * 2, 4 * H, out, None, D ** -0.5,
                            True, 0, picked, 5, ws, ibp.PAGED_WORKSPACE_BYTES)
    assert torch.equal(out, want) and c.status() == ibp.IBP_OK
    with pytest.raises(ibp.IbpError):
        ibp.ibp_paged_attention(c.handle, b.desc, got_q, 4 * H * D * 2, 4 * H, out, None, 0.125,
                                True, 0, None, 0, ws, 1024)
