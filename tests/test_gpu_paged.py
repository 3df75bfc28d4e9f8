"""The paged K/V cache (ibp_paged_*) against plain 64-bit implementations.

Pages lie in a shuffled order in their pool; memory that no token was written to
holds NaN; the page table's unused columns hold -1.  Bounds:

  unit roundoff u of the 16-bit type: 2^-11 (fp16), 2^-8 (bf16); fp32: e = 2^-24.
  append     the fp32 arithmetic of a channel is a handful of roundings and a sum of
             squares of D terms: relative error of each product at most (D + 16) e;
             then one rounding to 16 bits (or half the smallest subnormal of fp16).
  attention  a score is a product of D terms, each exact in fp32, summed in fp32 with
             truncation at worst: |ds| <= 2 D e scale sum |q||k| =: s_err, plus the
             scaling's and the exponential's roundings, 2^-20 |s| and 2^-20: every
             weight is off by a factor within 1 +- d, d = 2 (s_err + 2^-20 |s|max + 2^-20), and
             is rounded to 16 bits before it multiplies the values (u, or 2^-25 for a
             subnormal of fp16, against a sum of at least 1).  So
             |do| <= u |o| + (u + 2 d) sum p|v| + keys 2^-25 max|v| (fp16) + 2^-20 sum p|v|.
             lse: d / 2 + 2^-22 |lse| + 2^-20.
  bounds     exact (minima and maxima of 16-bit values).
  scores     2 D products exact in fp32, summed in fp32: 4 D e sum |q| max(|lo|, |hi|).
  selection  exact.
"""
import math

import numpy as np
import pytest
import torch

from lossless_invariant_bit_gb300 import ibp
from lossless_invariant_bit_gb300.paged import PagedCache
from lossless_invariant_bit_gb300.store import IbpStore
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F64 = torch.float64


class Setup:
    """A cache, a batch over it and its sequences' keys and values in order."""

    def __init__(self, q_lens, kv_lens, G=1, H=2, D=64, P=16, dtype=torch.float16, layout="rows",
                 seed=0, extra=3, max_q=None, poison=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g, self.G, self.H, self.D, self.P, self.dtype = g, G, H, D, P, dtype
        self.q_lens, self.kv_lens = q_lens, kv_lens
        need = [-(-n // P) for n in kv_lens]
        self.n_pages = sum(need) + extra
        cols = max(1, max(need))
        perm = torch.randperm(self.n_pages, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((len(kv_lens), cols + 1), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = perm[at:at + n]
            at += n
        self.table = table.to(DEV)[:, :cols]  # a stride of its own
        self.cols = cols
        shape = ((self.n_pages, P, H, D) if layout == "rows" else (self.n_pages, H, P, D))
        self.k = torch.full(shape, float("nan") if poison else 0.0, dtype=dtype, device=DEV)
        self.v = self.k.clone()
        if layout == "heads":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.K, self.V = [], []
        for s, n in enumerate(kv_lens):
            kk = torch.randn((n, H, D), generator=g, device=DEV).to(dtype)
            vv = torch.randn((n, H, D), generator=g, device=DEV).to(dtype)
            self.K.append(kk)
            self.V.append(vv)
            self.put(s)
        self.T = sum(q_lens)
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn((max(self.T, 1), H * G, D), generator=g, device=DEV).to(dtype)[:self.T]
        self.cache = PagedCache(H, D, P, self.n_pages, dtype, k=self.k, v=self.v)
        self.batch = self.cache.batch(self.table,
                                      torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                                      torch.tensor(self.starts, dtype=torch.int32, device=DEV),
                                      self.T, max_q or max(1, max(q_lens)))

    def put(self, s):
        n = self.kv_lens[s]
        pos = torch.arange(n, device=DEV)
        page = self.table[s, pos // self.P].long()
        self.k[page, pos % self.P] = self.K[s]
        self.v[page, pos % self.P] = self.V[s]

    def check_attention(self, out, lse, causal=True, window=0, scale=None, pages=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        u, G, e = U[self.dtype], self.G, 2.0 ** -24
        assert self.cache.status() == ibp.IBP_OK
        for s, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0:
                continue
            lo = self.starts[s]
            pos = torch.arange(L - n, L, device=DEV)[:, None]
            j = torch.arange(L, device=DEV)[None]
            for h in range(self.H):
                see = (j <= pos) if causal else torch.ones((n, L), dtype=torch.bool, device=DEV)
                if window:
                    see = see & (j > pos - window)
                if pages is not None:
                    pick = torch.zeros((n, self.cols + 1), dtype=torch.bool, device=DEV)
                    idx = pages[lo:lo + n, h].long()
                    pick.scatter_(1, torch.where(idx < 0, self.cols, idx.clamp(max=self.cols)),
                                  True)
                    see = see & pick[:, j[0] // self.P]
                see = see.repeat_interleave(G, 0)
                q = self.q[lo:lo + n, h * G:(h + 1) * G].reshape(n * G, self.D).to(F64)
                k, v = self.K[s][:, h].to(F64), self.V[s][:, h].to(F64)
                # what no row sees has no part in it, whatever it holds
                kz = torch.where(see.any(0)[:, None], k, 0.0)
                x = torch.where(see, q @ kz.T * scale, float("-inf"))
                absx = torch.where(see, q.abs() @ kz.abs().T * scale, 0.0)
                top = x.amax(1, keepdim=True) if L else torch.full((n * G, 1), -math.inf,
                                                                   device=DEV, dtype=F64)
                top = torch.where(top == -math.inf, 0.0, top)
                p = torch.exp(x - top)
                tot = p.sum(1, keepdim=True)
                p = p / torch.where(tot == 0, 1.0, tot)
                vz = torch.nan_to_num(v, 0.0, 0.0, 0.0)
                ref = p @ vz
                absv = p @ vz.abs()
                # infinities and NaN reach the rows that see them
                odd = torch.where(torch.isfinite(v), 0.0, v)
                for t in torch.nonzero((odd != 0).any(1)).flatten().tolist():
                    ref = ref + torch.where(see[:, t:t + 1], odd[t][None], 0.0)
                err_s = 2 * self.D * e * absx.amax(1, keepdim=True) if L else 0 * top
                smax = torch.where(see, x, 0.0).abs().amax(1, keepdim=True) if L else 0 * top
                d = 2 * (err_s + 2.0 ** -20 * smax + 2.0 ** -20)
                bound = u * ref.abs() + (u + 2 * d + 2.0 ** -20) * absv
                if self.dtype == torch.float16:
                    vm = torch.where(see.any(0)[:, None], vz.abs(), 0.0)
                    bound = bound + (L * 2.0 ** -25 * (vm.max() if L else 0.0) + 2.0 ** -25)
                got = out[lo:lo + n, h * G:(h + 1) * G].reshape(n * G, self.D).to(F64)
                fine = torch.isfinite(ref)
                assert torch.equal(fine, torch.isfinite(got)), (s, h)
                assert torch.equal(torch.isnan(ref), torch.isnan(got)), (s, h)
                inf = torch.isinf(ref)
                assert torch.equal(got[inf], ref[inf]), (s, h)
                diff = torch.where(fine, (got - ref).abs(), 0.0)
                assert bool((diff <= torch.where(fine, bound, 1.0)).all()), (
                    s, h, (diff - bound).max().item())
                ref_l = (top + torch.log(tot))[:, 0]
                got_l = lse[lo:lo + n, h * G:(h + 1) * G].reshape(n * G).to(F64)
                none = tot[:, 0] == 0
                assert torch.equal(none, got_l == -math.inf), (s, h)
                assert bool((got_l - ref_l)[~none].abs().le(
                    (d[:, 0] / 2 + 2.0 ** -22 * ref_l.abs() + 2.0 ** -20)[~none]).all()), (s, h)


def attend(st, **kw):
    out, lse = st.cache.attention(st.batch, st.q, lse=True, **kw)
    st.check_attention(out, lse, **kw)
    return out, lse


# ---------------------------------------------------------------- attention
# lengths about the blocks' (128 keys), the tiles' (16, 128 and 256 rows) and the pages' ends,
# none, one, fewer keys than new tokens (rows that see nothing)
STEPS = ([1, 1, 1, 1, 1, 1, 1, 0, 1], [1, 16, 127, 128, 129, 257, 700, 5, 0])
FEW = ([2, 3, 4, 1, 2, 0, 4], [2, 130, 300, 1, 1, 0, 257])
CHUNKS = ([17, 128, 129, 1, 300, 0, 40, 3], [17, 200, 129, 90, 431, 7, 30, 1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,P,layout", [(64, 16, "rows"), (128, 32, "heads"), (80, 8, "rows"),
                                        (16, 64, "heads"), (112, 256, "rows")])
@pytest.mark.parametrize("lens,G", [(STEPS, 1), (STEPS, 8), (STEPS, 16), (FEW, 4), (FEW, 3),
                                    (CHUNKS, 1), (CHUNKS, 5), (STEPS, 24)])
def test_attention(lens, G, D, P, layout, dtype):
    st = Setup(*lens, G=G, D=D, P=P, layout=layout, dtype=dtype, seed=G * 131 + D)
    attend(st)


@pytest.mark.parametrize("lens,G", [(FEW, 4), (CHUNKS, 2), (STEPS, 2)])
@pytest.mark.parametrize("window", [1, 7, 128, 200])
def test_attention_window(lens, G, window):
    for D, dtype in ((64, torch.bfloat16), (128, torch.float16)):
        attend(Setup(*lens, G=G, D=D, dtype=dtype, seed=window), window=window)


@pytest.mark.parametrize("lens,G", [(STEPS, 4), (FEW, 2), (CHUNKS, 3)])
def test_attention_without_mask(lens, G):
    attend(Setup(*lens, G=G, D=128, dtype=torch.bfloat16, P=32), causal=False, scale=0.2)


@pytest.mark.parametrize("q_lens,kv_lens,G,H,D", [
    ([1], [40000], 4, 1, 128),            # one row block cut over every CTA
    ([1, 1], [9001, 3], 1, 3, 64),
    ([5], [20011], 12, 1, 128),           # 60 rows: alternate blocks, cut
    ([40], [10007], 4, 1, 64),            # 160 rows, cut
    ([700, 1, 1], [5000, 4999, 2500], 7, 2, 128),  # whole and cut tiles, both kernels
    ([1] * 300, [1 + 37 * i % 400 for i in range(300)], 2, 1, 64),  # more sequences than threads
    ([20] * 200, [20 + 13 * i % 300 for i in range(200)], 1, 1, 128),
])
def test_attention_cut_tiles(q_lens, kv_lens, G, H, D):
    for dtype in (torch.float16, torch.bfloat16):
        attend(Setup(q_lens, kv_lens, G=G, H=H, D=D, dtype=dtype, seed=len(q_lens)))


@pytest.mark.parametrize("q_lens,kv_lens,G,H,window", [
    ([17] * 61, [17 + 5 * i for i in range(61)], 1, 3, 0),   # tiles of one to three blocks
    ([20] * 450, [20 + 7 * i % 200 for i in range(450)], 1, 1, 0),  # more than a CTA has threads
    ([90, 1, 45, 18], [90, 700, 1900, 18], 11, 2, 0),        # G that divides no tile
    ([150, 33], [4000, 50], 13, 1, 300),
])
def test_attention_of_many_short_tiles(q_lens, kv_lens, G, H, window):
    """Each tile stands for some blocks more than it has in the list that is cut
    into runs: runs end before a tile's first block, and with it."""
    for D, dtype in ((64, torch.float16), (128, torch.bfloat16)):
        attend(Setup(q_lens, kv_lens, G=G, H=H, D=D, dtype=dtype, seed=len(q_lens) + G),
               window=window)


def test_attention_large_scores_move_the_reference():
    """Keys that grow along the sequence: the running maximum outgrows every
    reference taken before, by far."""
    for q_lens, G in (([1], 4), ([130], 2)):
        st = Setup(q_lens, [1500], G=G, D=64, dtype=torch.bfloat16, seed=3)
        ramp = torch.linspace(0.1, 6.0, 1500, device=DEV)[:, None, None]
        st.K[0] = (st.K[0].float() * ramp).to(st.dtype)
        st.put(0)
        attend(st)


@pytest.mark.parametrize("q_lens,kv_lens,G", [([4, 3], [300, 131], 4), ([200, 33], [333, 260], 2),
                                              ([60], [400], 2)])
@pytest.mark.parametrize("window", [0, 40])
def test_infinities_and_nan_reach_only_rows_that_see_them(q_lens, kv_lens, G, window):
    """Values of the newest tokens are inf or NaN: earlier rows of the same tile
    do not see those tokens."""
    for dtype in (torch.float16, torch.bfloat16):
        st = Setup(q_lens, kv_lens, G=G, D=64, dtype=dtype, seed=11)
        for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
            for back, d, x in ((1, 3, math.inf), (n // 2 + 1, 9, -math.inf), (n, 17, math.nan),
                               (n + 20, 40, math.inf)):
                st.V[s][L - back, 0, d] = x
            st.put(s)
        attend(st, window=window)


def test_keys_that_are_nan_reach_only_rows_that_see_them():
    st = Setup([4, 150], [300, 260], G=4, D=64, dtype=torch.bfloat16, seed=12)
    out0, lse0 = st.cache.attention(st.batch, st.q, lse=True)
    for s, L in enumerate(st.kv_lens):
        st.K[s][L - 2, 0] = math.nan
        st.put(s)
    out, lse = st.cache.attention(st.batch, st.q, lse=True)
    for s, n in enumerate(st.q_lens):
        lo = st.starts[s]
        sees = torch.zeros(n, dtype=torch.bool, device=DEV)
        sees[n - 2:] = True
        for h in range(2):
            rows = slice(h * 4, h * 4 + 4)
            a, b = out[lo:lo + n, rows], out0[lo:lo + n, rows]
            if h == 0:
                assert bool(torch.isnan(a[sees]).all()) and torch.equal(a[~sees], b[~sees])
                assert torch.equal(lse[lo:lo + n, rows][~sees], lse0[lo:lo + n, rows][~sees])
            else:
                assert torch.equal(a, b)


def test_the_same_call_twice_gives_the_same_bits():
    st = Setup([300, 1, 1, 5], [3001, 4000, 77, 2000], G=8, D=128, dtype=torch.bfloat16)
    a = st.cache.attention(st.batch, st.q, lse=True)
    for _ in range(3):
        b = st.cache.attention(st.batch, st.q, lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_strided_queries_other_stream_and_graph():
    st = Setup([1, 140, 3], [900, 500, 64], G=2, D=64, dtype=torch.float16, seed=8)
    wide = torch.zeros((st.T, 3 * st.q.shape[1], st.D), dtype=st.dtype, device=DEV)
    wide[:, 4:8] = st.q
    ref = st.cache.attention(st.batch, st.q)
    assert torch.equal(st.cache.attention(st.batch, wide[:, 4:8]), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = st.cache.attention(st.batch, wide[:, 4:8], stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = st.cache.attention(st.batch, st.q)
    st.batch.kv_lens.copy_(torch.tensor([800, 400, 60], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, st.cache.attention(st.batch, st.q)) and not torch.equal(got, ref)


def test_pages_beyond_4_gib():
    """A pool whose offsets pass 32 bits: only its last pages are used."""
    n_pages = 9 * 2 ** 10  # 9216 pages of 256 tokens x 8 heads x 128 x 2 bytes = 4.5 GiB
    H, D, P = 8, 128, 256
    k = torch.empty((n_pages, P, H, D), dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    small = Setup([1, 40], [1000, 600], G=2, H=H, D=D, P=P, layout="rows", seed=4)
    first = n_pages - small.n_pages
    k[first:] = small.k
    v[first:] = small.v
    big = PagedCache(H, D, P, n_pages, torch.float16, k=k, v=v)
    table = torch.where(small.table >= 0, small.table + first, -1).contiguous()
    batch = big.batch(table, small.batch.kv_lens, small.batch.q_starts, small.T, 40)
    assert torch.equal(big.attention(batch, small.q),
                       small.cache.attention(small.batch, small.q))
    new = torch.randn((small.T, H, D), device=DEV).half()
    big.append(batch, new, new)
    small.cache.append(small.batch, new, new)
    assert torch.equal(k[first:].view(torch.int16), small.k.view(torch.int16))
    big.close()


# ---------------------------------------------------------------- lists of pages
@pytest.mark.parametrize("q_lens,kv_lens,G,D,P,n", [
    ([1, 1, 1], [4000, 100, 17], 4, 128, 16, 33),
    ([30, 1], [900, 1], 1, 64, 8, 7),
    ([5, 9], [1023, 1025], 24, 64, 64, 3),   # two blocks of 16 queries
    ([3], [2500], 16, 80, 256, 4),
    ([20], [400], 3, 128, 32, 40),           # every page, and more places than pages
])
def test_attention_over_lists(q_lens, kv_lens, G, D, P, n):
    for dtype in (torch.float16, torch.bfloat16):
        st = Setup(q_lens, kv_lens, G=G, D=D, P=P, dtype=dtype, seed=n)
        pages = torch.full((st.T, st.H, n), -1, dtype=torch.int32)
        rng = np.random.default_rng(n)
        for s, L in enumerate(kv_lens):
            for t in range(st.starts[s], st.starts[s + 1]):
                for h in range(st.H):
                    have = -(-L // P)
                    c = rng.permutation(have)[:n]
                    if t % 2:
                        c = np.sort(c)  # any order will do
                    pages[t, h, :len(c)] = torch.from_numpy(c.astype(np.int32))
        pages[0, 0] = -1  # a row that sees nothing
        attend(st, pages=pages.to(DEV))


def test_select_then_attend_over_every_page_equals_plain_attention():
    st = Setup([1, 6], [500, 300], G=2, D=64, P=16)
    pages = torch.arange(st.cols, dtype=torch.int32, device=DEV).expand(st.T, st.H, -1).contiguous()
    attend(st, pages=pages)


# ---------------------------------------------------------------- append
def rope_table(n, rot):
    half = rot // 2
    f = 10000.0 ** (-torch.arange(half, dtype=F64) / half)
    ang = torch.arange(n, dtype=F64)[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)


def turn(x, w, cs, rot, pairs, eps=1e-6):
    """(value, sum of the magnitudes of its terms) in 64 bits."""
    x = x.to(F64)
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.to(F64)
    y, m = x.clone(), x.abs().clone()
    if rot:
        i = torch.arange(rot // 2, device=DEV)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        c, s = cs[:, None, :rot // 2].to(F64), cs[:, None, rot // 2:].to(F64)
        u, v = x[..., a], x[..., b]
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        m[..., a] = (u * c).abs() + (v * s).abs()
        m[..., b] = (v * c).abs() + (u * s).abs()
    return y, m


def near(got, ref, mag, dtype, D):
    bound = U[dtype] * ref.abs() + (D + 16) * 2.0 ** -24 * 2 * mag + 2.0 ** -25
    d = (got.to(F64) - ref).abs()
    assert bool((d <= bound).all()), (d - bound).max().item()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,P,layout,rot", [(128, 16, "rows", 128), (64, 8, "heads", 32),
                                            (80, 32, "rows", 80), (96, 16, "rows", 16),
                                            (16, 256, "heads", 16), (128, 64, "rows", 0)])
@pytest.mark.parametrize("norm,pairs", [(True, False), (False, True), (True, True)])
def test_append(D, P, layout, rot, norm, pairs, dtype):
    q_lens, kv_lens = [1, 33, 0, 2, 64], [1, 40, 9, 17, 200]
    st = Setup(q_lens, kv_lens, G=3, D=D, P=P, layout=layout, dtype=dtype, seed=D, poison=False)
    H, T = st.H, st.T
    qkv = torch.randn((T, 3 * H + 2 * H, D), generator=st.g, device=DEV).to(dtype)
    q, k, v = qkv[:, :3 * H], qkv[:, 3 * H:4 * H], qkv[:, 4 * H:]
    qw = (1 + 0.1 * torch.randn(D, generator=st.g, device=DEV)).to(dtype) if norm else None
    kw = (1 + 0.1 * torch.randn(D, generator=st.g, device=DEV)).to(dtype) if norm else None
    cs = rope_table(200, rot) if rot else None
    before_k, before_v = st.k.clone(), st.v.clone()
    out = st.cache.append(st.batch, k, v, q=q, q_norm=qw, k_norm=kw, cos_sin=cs, pairs=pairs)
    assert st.cache.status() == ibp.IBP_OK
    wrote = torch.zeros((st.n_pages, P), dtype=torch.bool, device=DEV)
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        lo = st.starts[s]
        pos = torch.arange(L - n, L, device=DEV)
        page, slot = st.table[s, pos // P].long(), pos % P
        wrote[page, slot] = True
        near(out[lo:lo + n], *turn(q[lo:lo + n], qw, cs[pos] if rot else None, rot, pairs), dtype, D)
        near(st.k[page, slot], *turn(k[lo:lo + n], kw, cs[pos] if rot else None, rot, pairs), dtype,
             D)
        assert torch.equal(st.v[page, slot], v[lo:lo + n])
    assert torch.equal(st.k[~wrote], before_k[~wrote])
    assert torch.equal(st.v[~wrote], before_v[~wrote])
    # in place, without queries and without norms or rotation: copies
    st.cache.append(st.batch, k, v)
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        pos = torch.arange(L - n, L, device=DEV)
        assert torch.equal(st.k[st.table[s, pos // P].long(), pos % P],
                           k[st.starts[s]:st.starts[s] + n])
    buf = q.clone()
    assert st.cache.append(st.batch, k, v, q=buf, q_norm=qw, k_norm=kw, cos_sin=cs, pairs=pairs,
                           q_out=buf) is buf
    assert torch.equal(buf, out)


def test_append_many_tokens_and_heads():
    """Several rounds of heads per lane."""
    st = Setup([2500, 1], [2600, 9], G=8, H=5, D=128, dtype=torch.bfloat16, poison=False)
    q = torch.randn((st.T, 40, 128), generator=st.g, device=DEV).to(st.dtype)
    k = torch.randn((st.T, 5, 128), generator=st.g, device=DEV).to(st.dtype)
    w = torch.full((128,), 1.5, dtype=st.dtype, device=DEV)
    cs = rope_table(2600, 128)
    out = st.cache.append(st.batch, k, k, q=q, q_norm=w, cos_sin=cs)
    pos = torch.cat([torch.arange(100, 2600), torch.tensor([8])]).to(DEV)
    near(out, *turn(q, w, cs[pos], 128, False), st.dtype, 128)
    page = torch.cat([st.table[0, pos[:-1] // 16], st.table[1, pos[-1:] // 16]]).long()
    near(st.k[page, pos % 16], *turn(k, None, cs[pos], 128, False), st.dtype, 128)
    assert torch.equal(st.v[page, pos % 16], k)


# ---------------------------------------------------------------- bounds, scores, selection
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G,D,P", [(1, 64, 16), (4, 128, 8), (3, 80, 32), (16, 128, 64),
                                   (24, 64, 256), (7, 112, 16)])
def test_bounds_and_scores(G, D, P, dtype):
    q_lens, kv_lens = [1, 40, 0, 3, 9], [1, 700, 50, 33, 257]
    st = Setup(q_lens, kv_lens, G=G, D=D, P=P, dtype=dtype, seed=G)
    bounds = torch.full((st.n_pages, st.H, 2, D), 7.0, dtype=dtype, device=DEV)
    ref = bounds.clone()
    st.cache.update_bounds(st.batch, bounds)
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        for p in range((L - n) // P, (L - 1) // P + 1) if n else ():
            kk = st.K[s][p * P:(p + 1) * P]
            ref[st.table[s, p]] = torch.stack([kk.amin(0), kk.amax(0)], 1)
    assert torch.equal(bounds, ref)
    # every page's bounds, for the scores
    for s, L in enumerate(kv_lens):
        for p in range(-(-L // P)):
            kk = st.K[s][p * P:(p + 1) * P]
            bounds[st.table[s, p]] = torch.stack([kk.amin(0), kk.amax(0)], 1)
    scores = st.cache.page_scores(st.batch, st.q, bounds)
    assert st.cache.status() == ibp.IBP_OK
    for s, (n, L) in enumerate(zip(q_lens, kv_lens)):
        have = -(-L // P)
        for t in range(n):
            pos = L - n + t
            q = st.q[st.starts[s] + t].view(st.H, G, D).to(F64)
            b = bounds[st.table[s, :have].long()].to(F64)
            lo, hi = b[:, :, 0], b[:, :, 1]
            each = torch.maximum(q[None] * lo[:, :, None], q[None] * hi[:, :, None]).sum(-1)
            err = (q.abs()[None] * torch.maximum(lo.abs(), hi.abs())[:, :, None]).sum(-1)
            want = each.amax(2).T  # [H, pages]
            tol = 4 * D * 2.0 ** -24 * err.amax(2).T
            got = scores[st.starts[s] + t].to(F64)
            vis = pos // P + 1
            assert bool((got[:, vis:] == -math.inf).all())
            assert bool(((got[:, :vis] - want[:, :vis]).abs() <= tol[:, :vis]).all())
            # an upper bound of every product with the page's keys
            if t == 0:
                prod = torch.einsum("hgd,khd->hgk", q, st.K[s].to(F64)).amax(1)
                for p in range(vis):
                    assert bool((prod[:, p * P:(p + 1) * P].amax(1) <= want[:, p] + tol[:, p]).all())


def test_bounds_of_nan_keys_are_nan():
    st = Setup([3], [40], D=64, P=16)
    st.K[0][38, 1, 5] = math.nan
    st.put(0)
    bounds = torch.zeros((st.n_pages, 2, 2, 64), dtype=st.dtype, device=DEV)
    st.cache.update_bounds(st.batch, bounds)
    b = bounds[st.table[0, 2].long()]
    assert bool(torch.isnan(b[1, :, 5]).all()) and not bool(torch.isnan(b[0]).any())


def pick(scores, own, n):
    """The definition: the own page, then by score, equal ones by number."""
    x = [math.inf if math.isnan(v) else v for v in scores[:own + 1]]
    order = sorted(range(own + 1), key=lambda i: (i != own, -x[i], i))[:n]
    return sorted(order) + [-1] * max(0, n - own - 1)


@pytest.mark.parametrize("pages,rows,n", [(3, 1, 1), (300, 2, 7), (300, 2, 1), (300, 2, 300),
                                          (2047, 3, 100), (5000, 2, 33), (16384, 1, 700),
                                          (20000, 1, 64), (40, 3000, 6), (200, 2000, 9),
                                          (700, 1500, 100), (1800, 1300, 17), (30, 2500, 30)])
def test_select(pages, rows, n):
    """One or eight warps to a row, all they may hold, and rows that only the general form
    takes; scores of several kinds, some with many equal ones."""
    P, H = 8, 2
    L = pages * P - 3
    st = Setup([1], [L], D=16, P=P, H=H) if rows <= 3 else None
    if rows > 3:
        st = Setup([min(rows, L)], [L], D=16, P=P, H=H)
    elif rows > 1:
        st = Setup([rows], [L], D=16, P=P, H=H)
    g = torch.Generator(device=DEV)
    g.manual_seed(pages + n)
    T = st.T
    kinds = [
        torch.randn((T, H, st.cols), generator=g, device=DEV),
        torch.randint(-3, 4, (T, H, st.cols), generator=g, device=DEV).float() * 0.5,
        torch.zeros((T, H, st.cols), device=DEV),
        torch.exp(8 * torch.randn((T, H, st.cols), generator=g, device=DEV)),
    ]
    odd = kinds[0].clone()
    odd[torch.rand(odd.shape, generator=g, device=DEV) < 0.02] = math.inf
    odd[torch.rand(odd.shape, generator=g, device=DEV) < 0.02] = math.nan
    odd[torch.rand(odd.shape, generator=g, device=DEV) < 0.5] = -math.inf
    odd[:, :, ::7] = -0.0
    odd[:, :, 1::7] = 0.0
    kinds.append(odd)
    look = [0, T - 1] if T > 3 else list(range(T))
    for x in kinds:
        got = st.cache.select_pages(st.batch, x, n)
        for t in look + ([T // 2, T // 3] if T > 3 else []):
            own = (L - T + t) // P
            for h in range(H):
                assert got[t, h].tolist() == pick(x[t, h].tolist(), own, n), (t, h)
    assert st.cache.status() == ibp.IBP_OK


def test_select_rows_without_pages():
    st = Setup([3, 0, 2], [1, 0, 40], D=16, P=8)  # two tokens before the first position
    x = torch.randn((5, 2, st.cols), device=DEV)
    got = st.cache.select_pages(st.batch, x, 2)
    assert bool((got[:2] == -1).all())
    assert got[2].tolist() == [[0, -1]] * 2
    for t, own in ((3, 4), (4, 4)):
        for h in range(2):
            assert got[t, h].tolist() == pick(x[t, h].tolist(), own, 2)


# ---------------------------------------------------------------- refusals and data errors
def test_bad_page_ids_zero_the_rows_that_need_them():
    for q_lens, kv_lens, G in (([1, 1], [400, 300], 4), ([40, 150], [400, 300], 4)):
        st = Setup(q_lens, kv_lens, G=G, D=64, P=16, seed=2)
        want = st.cache.attention(st.batch, st.q)
        st.table[0, 3] = st.n_pages  # out of range
        out, lse = st.cache.attention(st.batch, st.q, lse=True)
        n = q_lens[0]
        assert st.cache.status() == ibp.IBP_ERANGE
        assert not bool(out[:n].any()) and bool((lse[:n] == -math.inf).all())
        assert torch.equal(out[n:], want[n:])
        assert st.cache.status() == ibp.IBP_OK
        # a window that does not reach the page needs it not
        a = st.cache.attention(st.batch, st.q, window=100)
        assert st.cache.status() == ibp.IBP_OK and bool(a[:n].any())
        st.table[0, 3] = -1
        st.cache.attention(st.batch, st.q)
        assert st.cache.status() == ibp.IBP_ERANGE


def test_bad_lengths_and_starts():
    st = Setup([2, 2, 2], [40, 50, 60], G=2, D=64, P=16, seed=2, poison=False)
    want = st.cache.attention(st.batch, st.q)
    st.batch.kv_lens[1] = 100000  # longer than its row of the table
    out, lse = st.cache.attention(st.batch, st.q, lse=True)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert not bool(out[2:4].any()) and bool((lse[2:4] == -math.inf).all())
    assert torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:])
    k0 = st.k.clone()
    new = torch.randn((6, 2, 64), device=DEV).half()
    q = st.cache.append(st.batch, new, new, q=st.q)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert not bool(q[2:4].any())
    changed = (st.k != k0).flatten(1).any(1)
    assert set(torch.nonzero(changed).flatten().tolist()) <= set(
        st.table[0].tolist() + st.table[2].tolist())
    st.batch.kv_lens[1] = 50
    st.batch.q_starts[1:3] = torch.tensor([4, 2], dtype=torch.int32)  # decrease
    st.cache.attention(st.batch, st.q)
    st.cache.select_pages(st.batch, torch.zeros((6, 2, st.cols), device=DEV), 2)
    st.cache.append(st.batch, new, new)
    st.cache.update_bounds(st.batch, torch.zeros((st.n_pages, 2, 2, 64), dtype=st.dtype, device=DEV))
    assert st.cache.status() == ibp.IBP_ERANGE
    # a rotation table that ends before a token's position
    st = Setup([1, 1], [40, 10], G=2, D=64, P=16, poison=False)
    cs = rope_table(20, 64)
    new = torch.randn((2, 2, 64), device=DEV).half()
    q = st.cache.append(st.batch, new, new, q=st.q, cos_sin=cs)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert not bool(q[0].any()) and bool(q[1].any())


def test_more_rows_than_the_batch_says_are_refused():
    st = Setup([9, 1], [40, 30], G=4, D=64, P=16, seed=2, max_q=4)
    out, _ = st.cache.attention(st.batch, st.q, lse=True)
    assert st.cache.status() == ibp.IBP_ERANGE
    assert bool(torch.isfinite(out[9:].float()).all())


def test_refusals():
    st = Setup([2], [40], G=2, D=64, P=16)
    c, b = st.cache, st.batch

    def status(call, code):
        with pytest.raises(ibp.IbpError) as e:
            call()
        assert e.value.status == code

    status(lambda: c.attention(b, st.q, scale=0.0), ibp.IBP_EINVAL)
    status(lambda: c.attention(b, st.q, scale=math.inf), ibp.IBP_EINVAL)
    status(lambda: c.attention(b, st.q, window=3, causal=False), ibp.IBP_EINVAL)
    pages = torch.zeros((2, 2, 1), dtype=torch.int32, device=DEV)
    status(lambda: c.attention(b, st.q, window=3, pages=pages), ibp.IBP_EINVAL)
    status(lambda: c.attention(b, st.q[:, :3], ), ibp.IBP_EINVAL)  # 3 heads on 2
    status(lambda: c.select_pages(b, torch.zeros((2, 2, st.cols), device=DEV), 0), ibp.IBP_EINVAL)
    k = torch.zeros((2, 2, 64), dtype=st.dtype, device=DEV)
    status(lambda: c.append(b, k, k, cos_sin=rope_table(40, 24)), ibp.IBP_EINVAL)
    status(lambda: c.append(b, k, k, eps=-1.0), ibp.IBP_EINVAL)
    status(lambda: c.append(b, k, k, q_norm=k[0, 0].contiguous()), ibp.IBP_EINVAL)  # no queries
    odd = torch.zeros(2 * 2 * 64 + 4, dtype=st.dtype, device=DEV)[4:].view(2, 2, 64)
    status(lambda: c.append(b, odd, odd), ibp.IBP_EALIGN)
    status(lambda: c.attention(b, torch.zeros(2 * 4 * 64 + 4, dtype=st.dtype,
                                              device=DEV)[4:].view(2, 4, 64)), ibp.IBP_EALIGN)
    for bad in (st.q.float(), st.q[:1], st.q[:, :, :32], st.q.transpose(0, 1)):
        with pytest.raises(ValueError):
            c.attention(b, bad)
    with pytest.raises(ValueError):
        c.attention(b, st.q, pages=pages.long())
    with pytest.raises(ValueError):
        c.update_bounds(b, torch.zeros((1, 2, 2, 64), dtype=st.dtype, device=DEV))
    with pytest.raises(ValueError):
        c.batch(st.table.long(), b.kv_lens, b.q_starts, 2, 2)
    for kw in (dict(head_dim=72), dict(head_dim=144), dict(page_tokens=12), dict(page_tokens=4),
               dict(page_tokens=512)):
        with pytest.raises(ibp.IbpError) as e:
            PagedCache(**{**dict(kv_heads=2, head_dim=64, page_tokens=16, n_pages=4), **kw})
        assert e.value.status == ibp.IBP_EINVAL
    with pytest.raises(ValueError):
        PagedCache(2, 64, 16, 4, torch.float32)
    # nothing to do is not an error
    empty = c.batch(st.table, b.kv_lens, torch.zeros(2, dtype=torch.int32, device=DEV), 0, 1)
    assert c.attention(empty, st.q[:0]).shape == (0, 4, 64)
    assert c.append(empty, k[:0], k[:0], q=st.q[:0]).shape == (0, 4, 64)


# ---------------------------------------------------------------- with the compressed store
def test_pages_go_to_a_compressed_host_store_and_come_back():
    """A sequence's keys and values leave their pages for compressed host slots
    (a token's keys are one row) and come back into other pages; a decode step over
    them gives the same bits."""
    H, D, P, G = 8, 128, 16, 4
    st = Setup([1, 1], [333, 200], G=G, H=H, D=D, P=P, layout="rows", poison=False, extra=30)
    want = st.cache.attention(st.batch, st.q)
    L, old = 333, st.table[0].clone()
    used = -(-L // P)
    rows = (old[:used].long()[:, None] * P + torch.arange(P, device=DEV)).flatten()[:L]
    free = sorted(set(range(st.n_pages)) - set(st.table[st.table >= 0].tolist()))[:used]
    for rows_of in (st.cache.key_rows, st.cache.value_rows):
        data = rows_of()
        store = IbpStore(H * D * 2, 256, L)
        try:
            seq = data[rows].contiguous()
            store.build(seq)
            slots, stored = store.compress(seq)
            data[rows] = 0  # the pages are someone else's now
            back = store.gather(slots, torch.arange(L, device=DEV))
            assert store.status() == ibp.IBP_OK
            new = (torch.tensor(free, device=DEV)[:, None] * P
                   + torch.arange(P, device=DEV)).flatten()[:L]
            data[new] = back
        finally:
            store.close()
    st.table[0, :used] = torch.tensor(free, dtype=torch.int32, device=DEV)
    assert torch.equal(st.cache.attention(st.batch, st.q), want)
