"""The paged K/V cache held in 8 bits and its page tables against plain 64-bit
implementations.

Pages lie in a shuffled order; slots that no token was written to hold NaN codes, scales
of pages that nothing uses the NaN byte.  Bounds, with e = 2^-24:

  append     keys: fp32 arithmetic of a handful of roundings and a sum of D squares, relative
             error d = (D + 16) e of each channel (of its rotation pair, at most |a| + |b|);
             then the nearest code, so |k - code * scale| <= half a step at the
             largest value it may have been + d.  A scale may be the next one where the largest
             magnitude is within d of 448 * 2^e.  Values: exact.
  attention  a score is a product of D terms exact in fp32 (11-bit queries, 4-bit codes),
             summed in fp32 with truncation at worst: 2 D e scale sum |q||k|, plus what bf16
             queries drop: 2^-38 of the row's largest q times sum |k|.  Scores, exponents and
             reference are added in fp32: (|s| + 130) 2^-23 more.  A weight is off by
             1 +- d and rounded to fp16: 2^-11 of it, or 2^-25 of the largest weight times
             scale, which multiplies codes of at most 448:
             |do| <= u |o| + (2^-11 + 2 d + 2^-20) sum p|v| + keys 2^-25 448 max(p scale).
             lse: d / 2 + 2^-22 |lse| + 2^-20.
  bounds     one rounding to the 16-bit type of an exact number: equal.
  tables     whole numbers: equal.
"""
import math

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp
from lossless_invariant_bit_gb300.paged import PagedCache
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

F64 = torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
NAN = 0x7F


def numbers():
    """What each code stands for."""
    return torch.arange(256, dtype=torch.uint8, device=DEV).view(E4M3).to(F64)


def two(e):
    """2^e of whole numbers, exactly."""
    return ((e.long() + 1023) << 52).view(F64)


class Setup:
    """A cache of random codes, a batch over it and its sequences' keys and values in order.

    spread: exponents of pages' scales lie in [-spread, spread]."""

    def __init__(self, q_lens, kv_lens, G=1, H=2, D=64, P=16, dtype=torch.float16, layout="rows",
                 seed=0, spread=3, max_q=None, extra=3):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g, self.G, self.H, self.D, self.P, self.dtype = g, G, H, D, P, dtype
        self.q_lens, self.kv_lens = q_lens, kv_lens
        need = [-(-n // P) for n in kv_lens]
        self.n_pages, self.cols = sum(need) + extra, max(1, max(need))
        perm = torch.randperm(self.n_pages, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((len(kv_lens), self.cols + 1), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = perm[at:at + n]
            at += n
        self.table = table.to(DEV)[:, :self.cols]  # a stride of its own
        shape = (self.n_pages, P, H, D) if layout == "rows" else (self.n_pages, H, P, D)
        self.codes = [torch.full(shape, NAN, dtype=torch.uint8, device=DEV) for _ in range(2)]
        if layout == "heads":
            self.codes = [c.transpose(1, 2) for c in self.codes]
        self.scales = [torch.full((self.n_pages, H), 255, dtype=torch.uint8, device=DEV)
                       for _ in range(2)]
        used = torch.cat([self.table[s, :n] for s, n in enumerate(need)]).long()
        for c, s in zip(self.codes, self.scales):
            x = (torch.randn((len(used), P, H, D), generator=g, device=DEV) * 60).clamp(-448, 448)
            c[used] = x.to(E4M3).view(torch.uint8)
            s[used] = torch.randint(127 - 6 - spread, 127 - 6 + spread + 1, (len(used), H),
                                    generator=g, device=DEV).to(torch.uint8)
        for s, n in enumerate(kv_lens):  # slots behind the last token
            if n % P:
                for c in self.codes:
                    c[self.table[s, n // P].long(), n % P:] = NAN
        self.T = sum(q_lens)
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn((max(self.T, 1), H * G, D), generator=g, device=DEV).to(dtype)[:self.T]
        self.cache = PagedCache(H, D, P, self.n_pages, dtype, k=self.codes[0].view(E4M3),
                                v=self.codes[1].view(E4M3), page_dtype=E4M3,
                                k_scales=self.scales[0].view(E8M0),
                                v_scales=self.scales[1].view(E8M0))
        self.batch = self.cache.batch(self.table,
                                      torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                                      torch.tensor(self.starts, dtype=torch.int32, device=DEV),
                                      self.T, max_q or max(1, max(q_lens)))

    def of(self, s, which):
        """Sequence s: its keys or values [L, H, D], and each one's scale [L, H]."""
        L = self.kv_lens[s]
        pos = torch.arange(L, device=DEV)
        page = self.table[s, pos // self.P].long()
        scale = two(self.scales[which][page].long() - 127)
        return numbers()[self.codes[which][page, pos % self.P].long()] * scale[..., None], scale

    def check(self, out, lse, causal=True, window=0, scale=None, pages=None, zero=(), status=0,
              weight=2.0 ** -11):
        """zero: rows (sequence, token) that could not be read; weight: the rounding of a weight
        (fp16's half step, where pages are made 16-bit ones first bf16's)."""
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        u, G, e = U[self.dtype], self.G, 2.0 ** -24
        assert self.cache.status() == status
        for s, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0:
                continue
            lo = self.starts[s]
            K, _ = self.of(s, 0)
            V, VS = self.of(s, 1)
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
                for z in zero:
                    if z[0] == s:
                        see[z[1]] = False
                see = see.repeat_interleave(G, 0)
                q = self.q[lo:lo + n, h * G:(h + 1) * G].reshape(n * G, self.D).to(F64)
                k, v = K[:, h], V[:, h]
                kz = torch.where(see.any(0)[:, None], k, 0.0)
                x = torch.where(see, q @ kz.T * scale, float("-inf"))
                kf = kz.nan_to_num(0.0)
                ax = torch.where(see, q.abs() @ kf.abs().T * scale, 0.0)
                drop = torch.where(see, q.abs().amax(1, keepdim=True) * kf.abs().sum(1)[None]
                                   * scale * 2.0 ** -38, 0.0)
                top = x.nan_to_num(float("-inf")).amax(1, keepdim=True) if L else \
                    torch.full((n * G, 1), -math.inf, device=DEV, dtype=F64)
                top = torch.where(top == -math.inf, 0.0, top)
                p = torch.exp(x - top)
                tot = p.sum(1, keepdim=True)
                p = p / torch.where(tot == 0, 1.0, tot)
                vz = v.nan_to_num(0.0)
                ref = p @ vz
                for t in torch.nonzero(torch.isnan(v).any(1)).flatten().tolist():
                    ref = ref + torch.where(see[:, t:t + 1] & torch.isnan(v[t])[None],
                                            float("nan"), 0.0)
                absv = p @ vz.abs()
                smax = torch.where(see, x, 0.0).abs().amax(1, keepdim=True) if L else 0 * top
                err = (2 * self.D * e * ax + drop).amax(1, keepdim=True) if L else 0 * top
                d = 2 * (err + (smax + 130) * 2.0 ** -23 + 2.0 ** -20)
                quantum = (torch.where(see, p * VS[:, h][None], 0.0).amax(1, keepdim=True) * 448
                           if L else 0 * top)
                bound = (u * ref.abs() + (weight + 2 * d + 2.0 ** -20) * absv
                         + L * 2.0 ** -25 * quantum)
                if self.dtype == torch.float16:
                    bound = bound + 2.0 ** -25
                got = out[lo:lo + n, h * G:(h + 1) * G].reshape(n * G, self.D).to(F64)
                big = ref.abs() > 65504.0 if self.dtype == torch.float16 else ref.abs() > 3e38
                nan = torch.isnan(ref)
                assert torch.equal(torch.isnan(got), nan), (s, h)
                fine = ~nan & ~big
                worst = ((got - ref).abs() - bound)[fine]
                assert worst.numel() == 0 or worst.max() <= 0, (s, h, worst.max())
                if lse is not None:
                    want = (top + torch.log(tot))[:, 0]
                    have = lse[lo:lo + n, h * G:(h + 1) * G].reshape(-1).to(F64)
                    some = tot[:, 0] > 0
                    assert torch.equal(have[~some & ~torch.isnan(tot[:, 0])],
                                       want[~some & ~torch.isnan(tot[:, 0])]), (s, h)
                    off = (have - want)[some].abs() - (
                        d[:, 0] / 2 + 2.0 ** -22 * want.abs() + 2.0 ** -20)[some]
                    assert off.numel() == 0 or off.max() <= 0, (s, h, off.max())


def attend(s, **kw):
    out, lse = s.cache.attention(s.batch, s.q, lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_lens,kv_lens,G,D,P", [
    ([1], [1], 1, 64, 16), ([1], [129], 1, 128, 16), ([1, 1, 1], [7, 1000, 33], 4, 128, 8),
    ([1] * 5, [300, 1, 64, 65, 2500], 1, 80, 64), ([1, 0, 1], [500, 20, 128], 16, 96, 128),
    ([2, 3, 1], [600, 77, 31], 5, 64, 32), ([4], [1027], 3, 16, 256), ([1], [40000], 2, 128, 16),
])
def test_step(q_lens, kv_lens, G, D, P, dtype):
    s = Setup(q_lens, kv_lens, G, 2, D, P, dtype)
    s.check(*attend(s))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_lens,kv_lens,G,D,P,layout", [
    ([33], [33], 1, 64, 16, "rows"), ([129], [400], 1, 128, 16, "heads"),
    ([300], [301], 2, 128, 32, "rows"), ([17, 1, 140], [900, 333, 141], 8, 128, 64, "rows"),
    ([70, 5], [70, 1200], 3, 80, 8, "heads"), ([513], [2000], 1, 48, 256, "rows"),
    ([1, 256, 2, 0, 31], [50, 256, 700, 9, 1000], 16, 64, 128, "rows"),
    ([40], [9000], 7, 112, 16, "rows"),
])
def test_chunk(q_lens, kv_lens, G, D, P, layout, dtype):
    s = Setup(q_lens, kv_lens, G, 2, D, P, dtype, layout)
    s.check(*attend(s))


BF16_WEIGHT = 2.0 ** -8  # half a step relative to the weight, as finfo(bf16).eps / 2


@pytest.mark.parametrize("q_lens,kv_lens,G,D,P,layout,window,causal", [
    ([1600], [1600], 1, 128, 16, "rows", 0, True), ([400, 801], [2001, 900], 4, 80, 8, "heads", 0, True),
    ([7, 1, 500], [300, 45, 513], 12, 112, 256, "rows", 0, True),
    ([900], [3000], 2, 128, 32, "heads", 77, True), ([333], [1111], 5, 96, 64, "rows", 0, False),
])
def test_long_chunks_of_bf16(q_lens, kv_lens, G, D, P, layout, window, causal):
    """Six tiles and more to a sequence and head: 16-bit pages in the workspace."""
    s = Setup(q_lens, kv_lens, G, 2, D, P, torch.bfloat16, layout)
    assert ibp.ibp_paged_workspace(s.cache.handle, s.batch.desc, 2 * G) > ibp.PAGED_WORKSPACE_BYTES
    out, lse = attend(s, window=window, causal=causal)
    s.check(out, lse, window=window, causal=causal, weight=BF16_WEIGHT)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = s.cache.attention(s.batch, s.q, window=window, causal=causal)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_long_chunks_of_bf16_bad_pages():
    """Pages that cannot be read and NaN in the others, through 16-bit pages."""
    for kv in (0, 1):
        s = Setup([500], [900], 4, 2, 128, 16, torch.bfloat16)
        s.codes[1][s.table[0, 40].long(), 3, 0, 5] = NAN  # a value: its head's channel alone
        good = attend(s)
        s.check(*good, weight=BF16_WEIGHT)
        at = s.table[0, 50].long()
        own = s.scales[kv][at, 1].clone()
        s.scales[kv][at, 1] = 255  # one head's page, from token 400 on
        out, lse = attend(s)
        assert s.cache.status() == ibp.IBP_ERANGE
        a, b = out.view(500, 2, 512).view(torch.int16), good[0].view(500, 2, 512).view(torch.int16)
        assert not out.view(500, 2, 512)[400:, 1].any()
        assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[:400], b[:400])
        assert (lse[400:, 4:] == -math.inf).all() and torch.equal(lse[:, :4], good[1][:, :4])
        s.scales[kv][at, 1] = own
        s.table[0, 50] = s.n_pages
        out, _ = attend(s)
        assert s.cache.status() == ibp.IBP_ERANGE
        assert not out[400:].any() and torch.equal(out[:400].view(torch.int16),
                                                   good[0][:400].view(torch.int16))


def test_small_workspace_of_long_chunks(monkeypatch):
    """Without the room the codes are multiplied: another rounding of the weights, no more."""
    from lossless_invariant_bit_gb300 import paged
    s = Setup([900], [3000], 2, 2, 128, 32, torch.bfloat16)
    s.check(*attend(s), weight=BF16_WEIGHT)
    with monkeypatch.context() as m:
        m.setattr(paged, "_MOST_WORKSPACE", 0)
        s.check(*attend(s))

    def none_left(*a):
        raise torch.OutOfMemoryError("none left")
    monkeypatch.setattr(paged, "_large_workspace", none_left)
    s.check(*attend(s))


def test_long_chunks_of_bf16_in_padded_batches():
    """Rows behind the last sequence stay; tokens without a position see nothing."""
    s = Setup([700, 900], [1000, 900], 4, 2, 128, 16, torch.bfloat16)
    want = s.cache.attention(s.batch, s.q)
    q = torch.cat([s.q, torch.full_like(s.q[:77], float("nan"))])
    out = torch.full_like(q, 3.0)
    b = s.cache.batch(s.table, s.batch.kv_lens, s.batch.q_starts, s.T + 77, 2000)
    s.cache.attention(b, q, out=out)
    assert torch.equal(out[:s.T], want) and bool((out[s.T:] == 3.0).all())
    assert s.cache.status() == 0
    s = Setup([700, 900], [1000, 600], 4, 2, 128, 16, torch.bfloat16)  # 300 of 900 have none
    got, lse = attend(s)
    s.check(got, lse, weight=BF16_WEIGHT)
    assert not got[700:1000].any() and bool((lse[700:1000] == -math.inf).all())


def test_long_chunks_of_bf16_in_wide_tables():
    """Columns that no sequence needs, more parts of pages than CTAs for a sequence."""
    s = Setup([300, 1, 400, 256, 300] * 8, [2500, 40, 400, 700, 3000] * 8, 8, 2, 128, 16,
              torch.bfloat16)
    wide = torch.full((40, 2000), -7, dtype=torch.int32, device=DEV)
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide
    s.batch = s.cache.batch(wide, s.batch.kv_lens, s.batch.q_starts, s.T, 400)
    assert ibp.ibp_paged_workspace(s.cache.handle, s.batch.desc, 16) > ibp.PAGED_WORKSPACE_BYTES
    out, lse = attend(s, window=2000)
    s.check(out, lse, window=2000, weight=BF16_WEIGHT)


def test_long_chunks_of_bf16_streams_threads_graphs():
    """The larger workspace: one for each stream, grown while calls are in flight, a graph's own."""
    import threading

    small = Setup([900], [1000], 2, 2, 128, 16, torch.bfloat16, seed=1)
    large = Setup([500, 900], [9000, 4000], 4, 2, 128, 16, torch.bfloat16, seed=2)
    want = [s.cache.attention(s.batch, s.q) for s in (small, large)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [[], []]

    def work(i, s):
        with torch.cuda.stream(side):
            outs[i].extend(s.cache.attention(s.batch, s.q) for _ in range(10))
        side.synchronize()

    ts = [threading.Thread(target=work, args=a) for a in enumerate((small, large))]
    for x in ts:
        x.start()
    for x in ts:
        x.join()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert len(o) == 10 and all(torch.equal(x, w) for x in o)
    graphs = []
    for s in (small, large):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.cache.attention(s.batch, s.q)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), w in zip(graphs, want):
            out.zero_()
            g.replay()
            s = small if w is want[0] else large
            beside = s.cache.attention(s.batch, s.q, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(out, w) and torch.equal(beside, w)
    assert small.cache.status() == 0 and large.cache.status() == 0


def test_many_short_tiles():
    """More tiles to a CTA than any of its rings is long, both kernels' at once."""
    q_lens = [17 + i % 30 if i % 3 else 1 + i % 4 for i in range(400)]
    kv_lens = [n + i * 7 % 50 for i, n in enumerate(q_lens)]
    for D in (64, 128):
        s = Setup(q_lens, kv_lens, 2, 6, D, 8, torch.bfloat16)
        out, lse = attend(s)
        s.check(out, lse)


def test_many_rows_of_one_token():
    """Few keys for each of many sequences: a tile of one block after the other."""
    for G, H, D in ((1, 8, 64), (8, 4, 128), (12, 4, 64)):
        s = Setup([1] * 300, [1 + i * 11 % 90 for i in range(300)], G, H, D, 16, torch.float16)
        out, lse = attend(s)
        s.check(out, lse)


@pytest.mark.parametrize("window", [1, 5, 128, 300])
@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 3], [700, 100], 2), ([90, 400], [700, 800], 4)])
def test_window(q_lens, kv_lens, G, window):
    s = Setup(q_lens, kv_lens, G, 2, 64, 16, torch.bfloat16)
    s.check(*attend(s, window=window), window=window)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 6], [70, 200]), ([200, 30], [200, 555])])
def test_not_causal(q_lens, kv_lens):
    s = Setup(q_lens, kv_lens, 3, 2, 128, 32, torch.float16)
    s.check(*attend(s, causal=False, scale=0.3), causal=False, scale=0.3)


@pytest.mark.parametrize("n", [1, 7, 40])
@pytest.mark.parametrize("D,P,G", [(128, 16, 4), (64, 32, 8), (80, 8, 20)])
def test_page_lists(n, D, P, G):
    s = Setup([1, 5, 37], [1, 333, 1000], G, 2, D, P, torch.bfloat16)
    pages = torch.full((s.T, 2, n), -1, dtype=torch.int32, device=DEV)
    r = torch.Generator()
    r.manual_seed(1)
    for i, (m, L) in enumerate(zip(s.q_lens, s.kv_lens)):
        for t in range(m):
            own = (L - m + t) // P
            for h in range(2):
                pick = torch.randperm(own + 3, generator=r)[:n].sort().values  # beyond it too
                pages[s.starts[i] + t, h, :len(pick)] = pick.to(torch.int32).to(DEV)
    s.check(*attend(s, pages=pages), pages=pages)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_lens,kv_lens,G,P", [([1, 2], [900, 130], 4, 8),
                                                ([150, 40], [600, 300], 2, 16),
                                                ([64], [800], 8, 64)])
def test_scales_that_differ_widely(q_lens, kv_lens, G, P, dtype):
    """Pages' scales over their whole range, queries to match: no page's values vanish
    beside another's."""
    s = Setup(q_lens, kv_lens, G, 2, 64, P, dtype, spread=0)
    g = s.g
    for w, spread in ((0, 12), (1, 49)):
        live = s.scales[w] != 255
        x = torch.randint(127 - spread, 127 + spread + 1, s.scales[w].shape, generator=g,
                          device=DEV).to(torch.uint8)
        s.scales[w].copy_(torch.where(live, x, s.scales[w]))
    s.q *= 2.0 ** -8
    s.check(*attend(s))


def test_one_huge_page_that_few_rows_see():
    """A page behind most rows' positions, with the largest scale: what other rows see
    keeps its bits."""
    s = Setup([128], [256], 2, 2, 64, 16, torch.bfloat16, spread=0)
    last = s.table[0, 15].long()
    for w in (0, 1):
        s.scales[w][last] = 177
    out, lse = attend(s)
    s.check(out, lse)
    assert bool(torch.isfinite(out[:100].float()).all())


@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 1], [200, 65], 4), ([3, 2], [150, 140], 2),
                                              ([130, 60], [300, 260], 4)])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_reaches_the_rows_that_see_it(which, q_lens, kv_lens, G):
    s = Setup(q_lens, kv_lens, G, 2, 64, 16, torch.float16)
    for seq, L in enumerate(kv_lens):
        for back, h, d in ((1, 0, 3), (2, 1, 60), (40, 0, 17)):
            pos = L - back
            s.codes[which][s.table[seq, pos // 16].long(), pos % 16, h, d] = 0xFF if d == 3 else NAN
    out, lse = attend(s)
    s.check(out, None)


@pytest.mark.parametrize("q_lens,kv_lens,G", [([1], [300], 4), ([2], [300], 4), ([100], [300], 4)])
@pytest.mark.parametrize("bad", ["id", "high id", "k", "v"])
def test_pages_that_cannot_be_read(bad, q_lens, kv_lens, G):
    """A page id or a scale out of range: rows that see it are zero, others are not."""
    s = Setup(q_lens, kv_lens, G, 2, 64, 16, torch.bfloat16)
    at = 17 if q_lens[0] > 2 else 4  # the page of positions 272 on, or one that all rows see
    page = int(s.table[0, at])
    keep = None
    if bad in ("id", "high id"):
        s.table[0, at] = -5 if bad == "id" else s.n_pages
    else:
        keep = s.scales["kv".index(bad)]
        keep[page] = torch.tensor([76, 178], dtype=torch.uint8, device=DEV)
    first = kv_lens[0] - q_lens[0]
    zero = [(0, t) for t in range(q_lens[0]) if first + t >= at * 16]
    out, lse = attend(s)
    for _, t in zero:
        assert bool((out[t] == 0).all()) and bool((lse[t] == -math.inf).all())
    if keep is not None:
        keep[page] = 127
    else:
        s.table[0, at] = page
    s.check(out, lse, zero=zero, status=ibp.IBP_ERANGE)


def test_rows_of_no_sequence_are_left_alone():
    s = Setup([3, 20], [40, 100], 2, 2, 64, 16)
    rows = s.T + 4
    q = torch.randn((rows, 4, 64), device=DEV).half()
    q[:s.T] = s.q
    out = torch.full_like(q, 7.0)
    b = s.cache.batch(s.table, s.batch.kv_lens, s.batch.q_starts, rows, 20)
    s.cache.attention(b, q, out=out)
    s.check(out, None)
    assert bool((out[s.T:] == 7.0).all())


def test_lengths_that_do_not_fit():
    """No keys, more new tokens than keys, a length beyond the table."""
    s = Setup([2, 4, 30], [40, 64, 100], 2, 2, 64, 16)
    lens = torch.tensor([0, 2, 101], dtype=torch.int32, device=DEV)
    lens[2] = s.cols * 16 + 1
    b = s.cache.batch(s.table, lens, s.batch.q_starts, s.T, 30)
    out, lse = s.cache.attention(b, s.q, lse=True)
    assert s.cache.status() == ibp.IBP_ERANGE
    assert bool((out[:2] == 0).all()) and bool((out[6:] == 0).all())
    assert bool((lse[:4] == -math.inf).all()) and bool((lse[6:] == -math.inf).all())
    # two of four tokens have positions
    assert bool((out[2:4] == 0).all()) and bool((out[4:6].abs().sum((1, 2)) > 0).all())


def test_strides_of_queries():
    s = Setup([1, 50], [100, 300], 4, 2, 128, 16, torch.bfloat16)
    wide = torch.zeros((s.T, 20, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 3:11] = s.q
    out, lse = s.cache.attention(s.batch, wide[:, 3:11], lse=True)
    s.check(out, lse)


def test_queries_of_all_magnitudes():
    """bf16 rows from the smallest to the largest magnitudes, and zero rows."""
    s = Setup([1, 40], [100, 200], 4, 2, 64, 16, torch.bfloat16, spread=0)
    f = torch.tensor([2.0 ** -126, 2.0 ** -60, 2.0 ** -10, 1.0, 2.0 ** 7, 0.0], device=DEV)
    i = torch.arange(s.T * 8, device=DEV) % 6
    s.q = (s.q.float() * f[i].view(s.T, 8, 1)).bfloat16()
    s.check(*attend(s))
    few = torch.zeros_like(s.q)
    few[..., 5] = 1e-30
    few[..., 6] = 3.0
    s.q = few
    s.check(*attend(s))


# ---------------------------------------------------------------- append
def rounded(x):
    """The nearest code's number, ties to the even code (|x| at most 448)."""
    codes = numbers()[:127]
    a = x.abs().contiguous()
    i = torch.searchsorted(codes, a).clamp(1, 126)
    below, above = a - codes[i - 1], codes[i] - a
    near = torch.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), codes[i - 1],
                       codes[i])
    return torch.where(x < 0, -near, near)


def need(m):
    """The exponent of the scale for a largest magnitude."""
    e = torch.full_like(m, -50).long()
    for c in range(-50, 50):
        e = torch.where(m > 448 * 2.0 ** c, c + 1, e)
    return e


def place(s, seq, pos):
    return s.table[seq, pos // s.P].long(), pos % s.P


def turned(x, cs, rot, pairs):
    y = x.clone()
    i0 = slice(0, rot, 2) if pairs else slice(0, rot // 2)
    i1 = slice(1, rot, 2) if pairs else slice(rot // 2, rot)
    c, n = cs[:, None, :rot // 2].to(F64), cs[:, None, rot // 2:].to(F64)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * n, b * c + a * n
    return y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_lens,kv_lens,H,D,P,rot,pairs,norm,layout", [
    ([1, 1, 1], [1, 17, 160], 2, 128, 16, 128, False, False, "rows"),
    ([1, 40, 3], [33, 40, 500], 3, 64, 8, 64, True, True, "rows"),
    ([100, 5], [203, 6], 2, 80, 32, 32, False, True, "heads"),
    ([300], [300], 1, 128, 256, 0, False, False, "rows"),
    ([700, 1], [900, 800], 5, 96, 128, 96, False, True, "rows"),
    ([9], [9], 4, 16, 64, 16, True, True, "rows"),
])
def test_append(q_lens, kv_lens, H, D, P, rot, pairs, norm, layout, dtype):
    G = 2
    s = Setup(q_lens, kv_lens, G, H, D, P, dtype, layout, spread=2)
    g = s.g
    x = torch.randn((s.T, (G + 2) * H, D), generator=g, device=DEV)
    x = (x * torch.exp(torch.randn((s.T, 1, 1), generator=g, device=DEV))).to(dtype)
    q, k, v = x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:]
    qw = kw = cs = None
    if norm:
        qw, kw = (1 + 0.1 * torch.randn((2, D), generator=g, device=DEV)).to(dtype)
    if rot:
        ang = torch.rand((max(kv_lens), rot // 2), generator=g, device=DEV) * 6.28
        cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    before = [c.clone() for c in s.codes], [c.clone() for c in s.scales]
    out = s.cache.append(s.batch, k, v, q=q, q_norm=qw, k_norm=kw, cos_sin=cs, pairs=pairs)
    assert s.cache.status() == 0
    table = numbers()
    touched = torch.zeros((s.n_pages, P), dtype=torch.bool, device=DEV)
    d = (D + 16) * 2.0 ** -24
    for seq, (n, L) in enumerate(zip(q_lens, kv_lens)):
        lo, pos = s.starts[seq], torch.arange(L - n, L, device=DEV)

        def formula(y, w):
            y = y[lo:lo + n].to(F64)
            if norm:
                y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.to(F64)
            size = y.abs()
            if rot:
                size = turned(size, cs[pos].abs() * torch.tensor(
                    [1.0] * (rot // 2) + [-1.0] * (rot // 2), device=DEV), rot, pairs).abs() \
                    + turned(size, cs[pos].abs(), rot, pairs).abs()
                y = turned(y, cs[pos], rot, pairs)
            return y, size

        want, size = formula(q, qw)
        err = (out[lo:lo + n].to(F64) - want).abs()
        assert bool((err <= U[dtype] * want.abs() + 2 * d * size + 2.0 ** -25).all())
        for w, (new, size) in enumerate((formula(k, kw), (v[lo:lo + n].to(F64), None))):
            for p in range((L - n) // P, (L - 1) // P + 1):
                at = int(s.table[seq, p])
                sel = (pos // P) == p
                y, slots = new[sel], (pos % P)[sel]
                touched[at, slots] = True
                tol = 0.0 if size is None else 2 * d * size[sel]
                t0 = int(slots[0])
                m = y.abs().amax((0, 2))
                low = high = need(m)
                if size is not None:
                    off = float(tol.max())
                    low, high = need(m - off), need(m + off)
                was = before[1][w][at].long() - 127
                if t0:
                    low, high = torch.maximum(low, was), torch.maximum(high, was)
                e = s.scales[w][at].long() - 127
                assert bool(((e >= low) & (e <= high)).all()), (seq, p, e, low, high)
                got = table[s.codes[w][at, slots].long()]
                y = y / two(e)[None, :, None]
                if size is None:
                    assert torch.equal(got, rounded(y)), (seq, p)
                else:  # between the codes of the values it may have been
                    t = tol / two(e)[None, :, None]
                    assert bool((got >= rounded((y - t).clamp(-448, 448))).all())
                    assert bool((got <= rounded((y + t).clamp(-448, 448))).all())
                if t0:
                    old = table[before[0][w][at, :t0].long()] * two(was - e)[None, :, None]
                    assert torch.equal(table[s.codes[w][at, :t0].long()], rounded(old)), (seq, p)
                    touched[at, :t0] = True
    for w in (0, 1):  # nothing else has changed
        assert torch.equal(s.codes[w][~touched], before[0][w][~touched])
        rest = ~touched.any(1)
        assert torch.equal(s.scales[w][rest], before[1][w][rest])


def test_append_of_what_is_not_finite():
    """Infinities and NaN become NaN codes and have no part in the scale; zeros, the smallest
    and the largest values keep to the scales' range."""
    s = Setup([6], [6], 1, 2, 64, 16, torch.bfloat16)
    x = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = math.inf, -math.inf, math.nan
    x[3, 0] = 3.5  # 448 * 2^-7
    x[4, 1] = 2.0 ** -70
    y = torch.zeros_like(x)
    y[0, 0], y[1, 1], y[2, 1] = 3e38, 2.0 ** 58, -0.0
    s.cache.append(s.batch, x, y)
    assert s.cache.status() == 0
    page = s.table[0, 0].long()
    k, v = (numbers()[c[page, :6].long()] for c in s.codes)
    assert s.scales[0][page].tolist() == [127 - 7, 127 - 50]
    assert torch.isnan(k).nonzero().tolist() == [[0, 0, 0], [1, 0, 1], [2, 0, 2]]
    assert bool((k[3, 0] == 448).all()) and bool((k[:, 1] == 0).all())
    assert s.scales[1][page].tolist() == [127 + 50, 127 + 50]
    assert bool((v[0, 0] == 448).all()) and bool((v[1, 1] == 256).all())
    assert s.codes[1][page, 2, 1].unique().tolist() == [0x80]


def test_append_that_outgrows_a_scale_again_and_again():
    """One token at a time into one page, each larger than the last."""
    H, D, P = 2, 32, 16
    cache = PagedCache(H, D, P, 2, torch.float16, page_dtype=E4M3)
    cache.k_scales.view(torch.uint8).fill_(255)
    cache.v_scales.view(torch.uint8).fill_(255)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    held = e = None
    for n in range(1, P + 1):
        x = (torch.randn((1, H, D), generator=g, device=DEV) * 1.7 ** n / 100).half()
        b = cache.batch(table, torch.tensor([n], dtype=torch.int32, device=DEV), starts, 1, 1)
        cache.append(b, x, x)
        new = need(x.to(F64).abs().amax((0, 2)))
        e2 = new if held is None else torch.maximum(e, new)
        if held is not None:
            held = rounded(held * two(e - e2)[None, :, None])
        y = rounded(x.to(F64) / two(e2)[None, :, None])
        held, e = y if held is None else torch.cat([held, y]), e2
        for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            assert torch.equal(scales.view(torch.uint8)[1].long() - 127, e)
            assert torch.equal(numbers()[codes.view(torch.uint8)[1, :n].long()], held)
    assert cache.status() == 0


def test_append_refuses_on_the_device():
    """Tokens without a position, beyond the rotation's rows, in pages out of range, beside a
    scale out of range: the status says so, the others are served."""
    s = Setup([4, 2, 3, 2], [2, 20, 40, 21], 1, 1, 64, 16, torch.float16)
    x = torch.ones((11, 1, 64), dtype=torch.float16, device=DEV)
    cs = torch.cat([torch.ones((39, 8)), torch.zeros((39, 8))], 1).to(DEV)
    s.table[1, 1] = s.n_pages
    s.scales[0][s.table[3, 1].long()] = 255
    before = [c.clone() for c in s.codes]
    q = s.cache.append(s.batch, x, x, q=x, cos_sin=cs)
    assert s.cache.status() == ibp.IBP_ERANGE
    n = numbers()
    for c, sc in zip(s.codes, s.scales):
        for seq, pos in ((0, 0), (0, 1), (2, 37), (2, 38), (3, 19), (3, 20)):
            page, slot = int(s.table[seq, pos // 16]), pos % 16
            assert bool((n[c[page, slot].long()] * two(sc[page].long() - 127) == 1.0).all())
    page = int(s.table[2, 2])
    for c, b in zip(s.codes, before):
        assert torch.equal(c[page, 7], b[page, 7])  # position 39: no row of the rotation
    assert q[:, 0, 0].tolist() == [0, 0, 1, 1, 0, 0, 1, 1, 0, 1, 1]


# ---------------------------------------------------------------- bounds
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 8), (80, 128), (16, 256)])
def test_bounds(D, P, dtype):
    s = Setup([1, 60, 0, 3], [1, 300, 50, 130], 1, 3, D, P, dtype)
    s.codes[0][s.table[3, 0].long(), 0, 1, 5] = NAN
    b = torch.full((s.n_pages, 3, 2, D), 7.0, dtype=dtype, device=DEV)
    want = b.clone()
    for seq, (n, L) in enumerate(zip(s.q_lens, s.kv_lens)):
        if n == 0:
            continue
        K = s.of(seq, 0)[0]
        for p in range((L - n) // P, (L - 1) // P + 1):
            x = K[p * P:min(L, (p + 1) * P)]
            want[int(s.table[seq, p]), :, 0] = x.amin(0).to(dtype)
            want[int(s.table[seq, p]), :, 1] = x.amax(0).to(dtype)
    s.cache.update_bounds(s.batch, b)
    assert s.cache.status() == 0
    assert torch.equal(b.nan_to_num(9.0), want.nan_to_num(9.0))
    # the scores take them
    sc = s.cache.page_scores(s.batch, s.q, b)
    pages = s.cache.select_pages(s.batch, sc, 2)
    assert pages.shape == (s.T, 3, 2) and s.cache.status() == 0


def test_bounds_of_a_scale_out_of_range():
    s = Setup([20], [20], 1, 1, 64, 16)
    s.scales[0][s.table[0, 1].long()] = 0
    b = torch.full((s.n_pages, 1, 2, 64), 7.0, dtype=torch.float16, device=DEV)
    s.cache.update_bounds(s.batch, b)
    assert s.cache.status() == ibp.IBP_ERANGE
    assert bool((b[s.table[0, 1].long()] == 7.0).all())
    assert not bool((b[s.table[0, 0].long()] == 7.0).any())


# ---------------------------------------------------------------- all of it
def test_the_calls_together_and_as_a_graph():
    """Tables, append and attention as a server runs them: prompts, steps, an end; the steps
    once more as one captured graph."""
    H, G, D, P, S = 2, 4, 64, 16, 5
    cache = PagedCache(H, D, P, 60, torch.bfloat16, page_dtype=E4M3)
    tables = cache.tables(S, 16)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    K, V = [[] for _ in range(S)], [[] for _ in range(S)]
    lens = [0] * S
    target = torch.zeros(S, dtype=torch.int32, device=DEV)

    def step(to):
        n = [max(0, b - a) for a, b in zip(lens, to)]
        target.copy_(torch.tensor(to, dtype=torch.int32))
        T = sum(n)
        batch, slots = tables.resize(target, T, max(n))
        k, v, q = (torch.randn((T, h, D), generator=g, device=DEV).bfloat16()
                   for h in (H, H, H * G))
        cache.append(batch, k, v)
        out = cache.attention(batch, q)
        assert cache.status() == 0
        at = 0
        for i in range(S):
            if to[i] < lens[i]:
                K[i], V[i] = K[i][:to[i]], V[i][:to[i]]
            if n[i] == 0:
                lens[i] = to[i]
                continue
            lens[i] = to[i]
            K[i] = list(K[i]) + list(k[at:at + n[i]])
            V[i] = list(V[i]) + list(v[at:at + n[i]])
            # what the pages hold: the nearest codes of what was appended
            pos = torch.arange(to[i], device=DEV)
            page = tables.page_table[i, pos // P].long()
            held = []
            for codes, scales, new in ((cache.k, cache.k_scales, K[i]),
                                       (cache.v, cache.v_scales, V[i])):
                f = two(scales.view(torch.uint8)[page].long() - 127)[..., None]
                x = numbers()[codes.view(torch.uint8)[page, pos % P].long()] * f
                new = torch.stack(list(new)).to(F64)
                # (half a step, or a subnormal's; twice, where a scale has grown)
                assert bool(((x - new).abs() <= new.abs() * 2.0 ** -4 + f * 2.0 ** -9).all())
                held.append(x)
            rows = cache.value_rows()[slots[at:at + n[i]]]  # the slots are the tokens' rows
            assert torch.equal(rows, cache.v.view(torch.uint8)[page, pos % P][to[i] - n[i]:]
                               .reshape(n[i], -1))
            x = q[at:at + n[i]].to(F64).view(n[i], H, G, D)
            sc = torch.einsum("nhgd,lhd->hgnl", x, held[0]) / 8
            hide = torch.ones((n[i], to[i]), dtype=torch.bool, device=DEV).triu(to[i] - n[i] + 1)
            w = sc.masked_fill(hide, -math.inf).softmax(-1)
            ref = torch.einsum("hgnl,lhd->nhgd", w, held[1])
            size = torch.einsum("hgnl,lhd->nhgd", w, held[1].abs())
            got = out[at:at + n[i]].to(F64).view(n[i], H, G, D)
            # scores below 40: their errors are below 2^-16 (the header's d)
            assert float(sc.abs().max()) < 40
            assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * size).all())
            at += n[i]

    step([100, 33, 1, 64, 17])
    for i in range(3):
        step([n + 1 for n in lens])
    step([lens[0] + 1, 0, lens[2] + 1, lens[3] + 1, lens[4] + 1])
    step([lens[0] + 1, 70, lens[2] + 1, lens[3] + 1, lens[4] + 5])
    free = int(tables.n_free)
    assert free == 60 - sum(-(-n // P) for n in lens)

    k, v, q = (torch.randn((S, h, D), generator=g, device=DEV).bfloat16() for h in (H, H, H * G))
    state = [t.clone() for t in (tables.kv_lens, tables.page_table, tables.free_pages,
                                 tables.n_free, cache.k.view(torch.uint8),
                                 cache.v.view(torch.uint8), cache.k_scales.view(torch.uint8),
                                 cache.v_scales.view(torch.uint8))]

    def reset():
        for t, x in zip((tables.kv_lens, tables.page_table, tables.free_pages, tables.n_free,
                         cache.k.view(torch.uint8), cache.v.view(torch.uint8),
                         cache.k_scales.view(torch.uint8), cache.v_scales.view(torch.uint8)),
                        state):
            t.copy_(x)
        target.copy_(tables.kv_lens)

    def one():
        target.add_(1)
        batch, _ = tables.resize(target, S, 1)
        cache.append(batch, k, v)
        return cache.attention(batch, q)

    reset()
    want = [one().clone() for _ in range(3)]
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
        side.synchronize()
        reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = one()
        reset()
        for x in want:
            graph.replay()
            side.synchronize()
            assert torch.equal(out, x)
    assert cache.status() == 0
    cache.close()


def test_calls_on_another_stream():
    s = Setup([1, 80], [300, 200], 4, 2, 128, 16, torch.float16)
    want = s.cache.attention(s.batch, s.q)
    torch.cuda.synchronize()
    for st in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        out = s.cache.attention(s.batch, s.q, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_the_same_call_gives_the_same_bits():
    s = Setup([1, 1, 200], [5000, 3, 3000], 4, 2, 128, 16, torch.bfloat16)
    a, la = s.cache.attention(s.batch, s.q, lse=True)
    for _ in range(3):
        b, lb = s.cache.attention(s.batch, s.q, lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_the_example():
    """The decode loop of examples/paged_decode.py over pages held in 8 bits."""
    import importlib.util
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "paged_decode", os.path.join(root, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    kw = dict(seqs=3, prompt=300, chunk=128, steps=5, hidden=256, q_heads=8, kv_heads=2, dim=64,
              bits=8)
    full, few, ratio, same, _ = m.run(pick=1000, **kw)
    assert same and 0 < ratio <= 1.0
    for x in (full, few):
        assert x.shape == (5, 3, 256) and bool(torch.isfinite(x.float()).all())
    b = m.run(pick=0, **kw)
    assert torch.equal(full, b[0])
    # every page selected: the same sums in another order, two roundings to bf16 on either
    # side of a projection
    d = (few.double() - b[1].double()).norm() / b[1].double().norm()
    assert d < 2.0 ** -7


def test_threads_on_one_stream():
    """Calls of two threads on one stream, each with its own cache and tables."""
    import threading

    def work(seed, out):
        s = Setup([1, 1], [300, 70], 4, 2, 64, 16, torch.float16, seed=seed)
        out.extend(s.cache.attention(s.batch, s.q) for _ in range(20))
        torch.cuda.synchronize()
        assert s.cache.status() == 0
        out.append(s)

    outs = [[], []]
    ts = [threading.Thread(target=work, args=(i, o)) for i, o in enumerate(outs)]
    for x in ts:
        x.start()
    for x in ts:
        x.join()
    for o in outs:
        s = o.pop()
        assert len(o) == 20 and all(torch.equal(x, o[0]) for x in o)
        s.check(o[0], None)
