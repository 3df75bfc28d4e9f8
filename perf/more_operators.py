"""The paged K/V cache held in 8 bits: cases, inputs, plain forms and 64-bit values.

Half the bytes of a 16-bit cache hold the same tokens, or twice the tokens fit: a page's
keys (and values) of one head are e4m3 codes with one scale, a power of two (E8M0), and
stand for code * scale.  Four operators keep and read such a cache, each reached
through `PagedCache` and its page tables:

  tables   sequences' lengths change: pages come from the list of free ones or go back
           to it, and each new token gets its row of the pages (block tables and slot maps)
  append   a step's keys and values, normalised and rotated on the way, into their pages'
           codes; where a page's values outgrow its scale, the codes it holds are rescaled
  bounds   the smallest and largest key of each channel of the pages that were appended to
  attend   a ragged batch of new tokens (one of a sequence that is being answered, many of
           a prompt's chunk) over everything in its pages, or over listed pages alone

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
LOW, HIGH = -50, 50  # exponents of scales


# ---------------------------------------------------------------- cases
def _case(name, op, seqs, q_max, kv_max, q_heads, kv_heads, dim, page, dtype, lens=0, **more):
    c = {"op": op, "seqs": seqs, "q_max": q_max, "kv_max": kv_max, "q_heads": q_heads,
         "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "lens": lens,
         "layout": "rows"}
    c.update(more)
    if name:
        c["name"] = name
    return c


def _tables(name, seqs, q_max, kv_max, page, lens, ended):
    c = {"op": "tables", "seqs": seqs, "q_max": q_max, "kv_max": kv_max, "page": page,
         "lens": lens, "ended": ended}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the 20 sequences of the K/V workload take 5 drafted tokens each, and give them back
        # when none was accepted: the tables of a decode step
        _tables("tables_step", 20, 5, 1984, 16, 0, False),
        # 250 sequences of up to 32768 tokens: about a third has ended, its pages go back,
        # and new prompts take their places
        _tables("tables_prompts", 250, 32768, 32768, 16, 3, True),
        # one token of each of the 20 sequences of the K/V workload (32 heads of 128, fp16),
        # rotated, without norms: a decode step's append, most of it into pages in use
        _case("append_step", "append", 20, 1, 1984, 32, 32, 128, 16, "fp16", lens=1,
              norm=False, rot=128, pairs=False),
        # prompts of odd lengths, 64 query heads on 8 K/V heads, with the norms of each head:
        # the append of a prefill step
        _case("append_prompt", "append", 11, 1531, 4000, 64, 8, 128, 32, "bf16", lens=5,
              norm=True, rot=128, pairs=False),
        # the newest page of 16 long sequences
        _case("bounds_step", "bounds", 16, 1, 32768, 32, 8, 128, 16, "bf16"),
        # every page of prompts of odd lengths
        _case("bounds_prompt", "bounds", 9, 5003, 5003, 16, 8, 128, 32, "fp16", lens=3),
        # one user, a short conversation: latency
        _case("attend_one", "attend", 1, 1, 517, 32, 32, 128, 16, "fp16", window=0, pick=0),
        # the K/V workload's decode step: 20 sequences of 1920 + 64 tokens, 32 heads of 128
        _case("attend_step", "attend", 20, 1, 1984, 32, 32, 128, 16, "fp16", window=0, pick=0),
        # a server's mixed batch: sequences that are being answered beside chunks of prompts,
        # odd lengths, heads of 64, a sliding window
        _case("attend_mixed", "attend", 24, 333, 6001, 32, 4, 64, 32, "bf16", lens=7,
              window=2500, pick=0),
        # chunked prefill: 2048 new tokens of 8192, 64 query heads on 8
        _case("attend_chunk", "attend", 1, 2048, 8192, 64, 8, 128, 64, "bf16", window=0, pick=0,
              layout="heads"),
        # 16 long sequences, one token each, over 128 pages of 16 tokens out of up to 2048
        _case("sparse_step", "attend", 16, 1, 32768, 32, 8, 128, 16, "bf16", window=0, pick=128),
        # tokens of a chunk, each over its own 24 pages of 32
        _case("sparse_chunk", "attend", 2, 119, 4099, 32, 4, 128, 32, "fp16", lens=4, window=0,
              pick=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("tables", "append", "append", "bounds", "attend", "attend", "attend",
                         "sparse"))
        page = rng.choice((8, 16, 16, 32, 64, 128))
        if op == "tables":
            ended = rng.random() < 0.5
            kv_max = _log(rng, 2, 65536)
            c = _tables(None, _log(rng, 1, 600), kv_max if ended else _log(rng, 1, min(kv_max, 64)),
                        kv_max, page, rng.randint(1, 999), ended)
            if sum(_lens(c)[1]) > 4.0e6:
                continue
            return c
        kv_heads = rng.choice((1, 2, 3, 4, 8, 8, 16, 32))
        group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
        seqs = _log(rng, 1, 64)
        q_max = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        kv_max = q_max + _log(rng, 1, 32768)
        c = _case(None, "attend" if op == "sparse" else op, seqs, q_max, kv_max, kv_heads * group,
                  kv_heads, rng.choice((64, 80, 96, 128, 128)), page, rng.choice(("bf16", "fp16")),
                  lens=rng.randint(0, 999), layout=rng.choice(("rows", "heads")))
        if c["q_heads"] > 128:
            continue
        if op == "append":
            c["norm"], c["pairs"] = rng.random() < 0.5, rng.random() < 0.5
            c["rot"] = rng.choice((0, c["dim"] // 32 * 16, c["dim"] // 16 * 16))
        if op in ("attend", "sparse"):
            c["pick"] = _log(rng, 1, 256) if op == "sparse" else 0
            c["window"] = 0 if op == "sparse" or rng.random() < 0.6 else _log(rng, 1, kv_max)
        w = work(c)
        pool = sum(-(-n // page) for n in _lens(c)[1]) * page * kv_heads * c["dim"] * 2
        tokens = sum(_lens(c)[0])
        plain = {"append": 0, "bounds": 0,
                 "attend": 4 * seqs * q_max * kv_max * c["q_heads"],
                 "sparse": 4 * tokens * kv_heads * c.get("pick", 0) * page * c["dim"]}[op]
        if w["flops"] > 4.4e11 or w["bytes"] > 6.0e8 or pool > 3e9 or plain > 1.2e10:
            continue
        return c


def _lens(c):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    if not c["lens"]:
        return [c["q_max"]] * c["seqs"], [c["kv_max"]] * c["seqs"]
    r = random.Random(c["lens"])
    q, kv = [], []
    for i in range(c["seqs"]):
        if c["op"] == "tables" and c["ended"]:
            n = l = c["kv_max"] if i == 0 else r.randint(1, c["kv_max"])
            if i and r.random() < 0.67:
                n = 0  # goes on
        elif c["op"] == "bounds" and c["q_max"] == c["kv_max"]:
            n = l = c["kv_max"] if i == 0 else r.randint(1, c["kv_max"])
        else:
            n = c["q_max"] if i == 0 else 1 if r.random() < 0.5 else r.randint(1, c["q_max"])
            l = c["kv_max"] if i == 0 else r.randint(max(n, c["kv_max"] // 8), c["kv_max"])
        q.append(n)
        kv.append(l)
    return q, kv


def work(c):
    """Bytes that have to be read and written and operations that have to be done."""
    q, kv = _lens(c)
    T, P = sum(q), c["page"]
    if c["op"] == "tables":
        # the pages that come and go, read and written each time, the new tokens' rows, and
        # lengths old and new of both calls
        if c["ended"]:
            pages = sum(-(-l // P) for n, l in zip(q, kv) if n)
        else:
            pages = sum(-(-(l + n) // P) - -(-l // P) for n, l in zip(q, kv))
        return {"bytes": 16 * pages + 8 * T + 2 * 12 * c["seqs"], "flops": 4 * T + 2 * pages}
    D, H = c["dim"], c["kv_heads"]
    G = c["q_heads"] // H
    rows = 2 * T * D  # bytes of one head of every token, in 16 bits
    touched = sum((l - 1) // P - (l - n) // P + 1 for n, l in zip(q, kv))
    if c["op"] == "append":
        n = 2 * rows * c["q_heads"] + 3 * rows * H + 4 * T * c["rot"] + 4 * touched * H
        return {"bytes": n, "flops": (4 * c["norm"] + 3 * bool(c["rot"])) * T * D * (c["q_heads"] + H)
                + 4 * T * D * H}
    if c["op"] == "bounds":
        held = sum(l - (l - n) // P * P for n, l in zip(q, kv))
        return {"bytes": held * H * D + touched * H * (4 * D + 1), "flops": 2 * held * H * D}
    keys = pairs = 0
    if c["pick"]:
        for n, l in zip(q, kv):
            mine = [min((l - n + i) // P, c["pick"] - 1) * P + (l - n + i) % P + 1
                    for i in range(n)]
            pairs += sum(mine)
            keys += min(l, sum(mine))
        more = 4 * T * H * c["pick"]
    else:
        win = c["window"] or 1 << 62
        for n, l in zip(q, kv):
            first = l - n  # position of the first new token
            pairs += sum(min(first + i + 1, win) for i in range(n))
            keys += l - max(0, first + 1 - win)
        more = 0
    return {"bytes": 2 * rows * c["q_heads"] + 4 * T * c["q_heads"] + 2 * keys * H * D
            + 2 * keys * H // P + more, "flops": 4 * D * c["q_heads"] * pairs}


# ---------------------------------------------------------------- inputs
class State:
    pass


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _need(m):
    """The smallest exponent e with m <= 448 * 2^e, of those that scales have."""
    f, k = torch.frexp(m)
    e = torch.where(f <= 0.875, k - 9, k - 8)
    return torch.where(m == 0, LOW, e).clamp(LOW, HIGH).to(torch.int32)


def _two(e):
    """2^e exactly, of whole numbers (inf for 128: a scale that is NaN)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, e):
    """x / 2^e as e4m3, the largest code where it is larger, NaN where it is not finite."""
    y = (x.float() * _two(-e)).clamp(-448.0, 448.0)
    return torch.where(torch.isfinite(x), y, float("nan")).to(E4M3).view(torch.uint8)


def prepare(c, seed):
    s = State()
    s.case = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, kv = _lens(c)
    P = c["page"]
    if c["op"] == "tables":
        return _prepare_tables(s, c, g, q, kv)
    dt = DTYPES[c["dtype"]]
    H, D = c["kv_heads"], c["dim"]
    T = sum(q)
    need = [-(-n // P) for n in kv]
    cols = max(need)
    n_pages = sum(need) + max(2, sum(need) // 16)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    lens = torch.tensor(need, device="cuda")
    at = (torch.cumsum(lens, 0) - lens)[:, None] + torch.arange(cols, device="cuda")[None]
    live = torch.arange(cols, device="cuda")[None] < lens[:, None]
    # columns that a sequence does not use hold no page
    s.table = torch.where(live, perm[at.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    s.kv_lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s.q_starts = torch.tensor([0] + q, device="cuda").cumsum(0).to(torch.int32)
    s.T, s.n_pages, s.cols = T, n_pages, cols
    # what the pages hold: for an append the tokens before the new ones, else all; memory
    # that no token has been written to, and the scales of free pages, hold what they may (NaN)
    free = torch.ones(n_pages, dtype=torch.bool, device="cuda")
    free[s.table[live].long()] = False
    hole = free[:, None].repeat(1, P)
    pos = torch.arange(cols * P, device="cuda").view(cols, P)
    held = s.kv_lens.long()
    if c["op"] == "append":
        held = held - torch.tensor(q, device="cuda")
    empty = (pos[None] >= held[:, None, None])[live]
    hole[s.table[live].long()] = empty
    shape = (n_pages, P, H, D) if c["layout"] == "rows" else (n_pages, H, P, D)
    chan = torch.exp(0.3 * _rand(g, H, D))
    for name, by in (("k", chan), ("v", 1.0)):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        if c["layout"] == "heads":
            codes = codes.transpose(1, 2)
        scales = torch.empty((n_pages, H), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (P * H * D))
        for lo in range(0, n_pages, step):
            x = _rand(g, min(step, n_pages - lo), P, H, D) * by
            none = hole[lo:lo + step]
            x[none] = 0.0
            e = _need(x.abs().amax((1, 3)))
            y = _codes(x, e[:, None, :, None])
            y[none] = 0x7F
            codes[lo:lo + step] = y
            scales[lo:lo + step] = (e + 127).to(torch.uint8)
        scales[hole.all(1)] = 0xFF
        setattr(s, name, codes)
        setattr(s, name + "_scales", scales)
    # a step's projections come as one matrix: queries, keys and values side by side
    if c["op"] == "append":
        qkv = _rand(g, T, c["q_heads"] + 2 * H, D).to(dt)
        s.q = qkv[:, :c["q_heads"]]
        s.k_new = qkv[:, c["q_heads"]:c["q_heads"] + H]
        s.v_new = qkv[:, c["q_heads"] + H:]
        s.q_norm = s.k_norm = s.cos_sin = None
        if c["norm"]:
            s.q_norm = (1 + 0.1 * _rand(g, D)).to(dt)
            s.k_norm = (1 + 0.1 * _rand(g, D)).to(dt)
        if c["rot"]:
            half = c["rot"] // 2
            freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
            ang = torch.arange(c["kv_max"], device="cuda", dtype=torch.float64)[:, None] * freq
            s.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
    elif c["op"] == "bounds":
        s.bounds = torch.zeros((n_pages, H, 2, D), dtype=dt, device="cuda")
    else:
        s.q = _rand(g, T, c["q_heads"], D).to(dt)
        s.pages = _lists(s, g) if c["pick"] else None
    if own:
        from lossless_invariant_bit_gb300.paged import PagedCache

        s.cache = PagedCache(H, D, P, n_pages, dt, k=s.k.view(E4M3), v=s.v.view(E4M3),
                             page_dtype=E4M3, k_scales=s.k_scales.view(E8M0),
                             v_scales=s.v_scales.view(E8M0))
        s.batch = s.cache.batch(s.table, s.kv_lens, s.q_starts, T, c["q_max"])
    return s


def _lists(s, g):
    """For each token and K/V head its own page and others at random, ascending, -1 behind."""
    c = s.case
    _, pos = _places(s)
    newest = (pos // c["page"])[:, None, None]
    j = torch.arange(s.cols, device="cuda")
    x = torch.rand((s.T, c["kv_heads"], s.cols), generator=g, device="cuda")
    x = torch.where(j > newest, -1.0, torch.where(j == newest, 2.0, x))
    top = torch.topk(x, min(c["pick"], s.cols), dim=-1)
    order = torch.where(top.values < 0, 1 << 30, top.indices).sort(-1).values
    out = torch.where(order == 1 << 30, -1, order).to(torch.int32)
    missing = c["pick"] - out.shape[-1]
    return torch.cat([out, out.new_full((*out.shape[:-1], missing), -1)], -1).contiguous()


def _prepare_tables(s, c, g, q, kv):
    P, S = c["page"], c["seqs"]
    low = torch.tensor([0 if c["ended"] and n else l for n, l in zip(q, kv)], device="cuda")
    high = torch.tensor([l if c["ended"] else l + n for n, l in zip(q, kv)], device="cuda")
    s.low, s.high = low.to(torch.int32), high.to(torch.int32)
    most = -(-high // P)
    s.cols = int(most.max())
    s.n_pages = int(most.sum()) + max(2, int(most.sum()) // 16)
    s.T = sum(q)
    # as it is when the pass begins: with the sequences that will end, or without new tokens
    s.kv_lens = (s.high if c["ended"] else s.low).clone()
    have = -(-s.kv_lens.long() // P)
    perm = torch.randperm(s.n_pages, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(s.cols, device="cuda")
    at = (torch.cumsum(have, 0) - have)[:, None] + j
    s.table = torch.where(j < have[:, None], perm[at.clamp(max=s.n_pages - 1)], -1)
    s.table = s.table.to(torch.int32).contiguous()
    used = int(have.sum())
    s.free = torch.full((s.n_pages,), -1, dtype=torch.int32, device="cuda")
    s.free[:s.n_pages - used] = perm[used:]
    s.n_free = torch.tensor([s.n_pages - used], dtype=torch.int32, device="cuda")
    s.slots = torch.empty(s.T, dtype=torch.int64, device="cuda")
    if own:
        from lossless_invariant_bit_gb300.paged import PagedCache

        s.cache = PagedCache(1, 16, P, s.n_pages, torch.bfloat16, page_dtype=E4M3)
        s.tables = s.cache.tables(S, s.cols)
        s.tables.page_table.copy_(s.table)
        s.tables.kv_lens.copy_(s.kv_lens)
        s.tables.free_pages.copy_(s.free)
        s.tables.n_free.copy_(s.n_free)
    return s


# ---------------------------------------------------------------- plain forms
def _places(s):
    """Each new token's sequence and position."""
    t = torch.arange(s.T, device="cuda")
    seq = torch.searchsorted(s.q_starts.long(), t, right=True) - 1
    starts = s.q_starts.long()
    return seq, s.kv_lens.long()[seq] - starts[seq + 1] + t


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, cs, rot, pairs):
    if not rot:
        return x
    c, n = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _write(s, codes, scales, x, seq, pos):
    """x [T, H, D] into the pages' codes, under scales that hold them and what was there."""
    P = s.case["page"]
    page, slot = s.table[seq, pos // P].long(), pos % P
    m = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    most = torch.zeros(scales.shape, device="cuda")
    most.scatter_reduce_(0, page[:, None].expand_as(m), m, "amax")
    starts = s.q_starts.long()
    first = s.kv_lens.long() - (starts[1:] - starts[:-1])
    mine = s.table.gather(1, (first // P)[:, None]).long()[:, 0]  # each sequence's first page
    older = (first % P > 0)[:, None]
    was = scales.to(torch.int32) - 127
    e = _need(most)
    e[mine] = torch.where(older, torch.maximum(e[mine], was[mine]), e[mine])
    # what those pages hold already, under the new scale
    c = codes[mine].view(E4M3).float()
    down = torch.where(older, was[mine] - e[mine], 0)
    c = (c * _two(down)[:, None, :, None]).to(E4M3).view(torch.uint8)
    kept = torch.arange(P, device="cuda")[None, :] < (first % P)[:, None]
    codes[mine] = torch.where(kept[..., None, None], c, codes[mine])
    codes[page, slot] = _codes(x, e[page][..., None])
    scales[page] = (e[page] + 127).to(torch.uint8)


def _append(s):
    c = s.case
    seq, pos = _places(s)
    cs = s.cos_sin[pos] if c["rot"] else None
    q = _rotate(_norm(s.q, s.q_norm), cs, c["rot"], c["pairs"]).to(s.q.dtype)
    k = _rotate(_norm(s.k_new, s.k_norm), cs, c["rot"], c["pairs"])
    _write(s, s.k, s.k_scales, k, seq, pos)
    _write(s, s.v, s.v_scales, s.v_new.float(), seq, pos)
    return _cache_of(s, q)


def _cache_of(s, q):
    """What an append leaves: the queries, and codes and scales as the numbers they are."""
    return (q, s.k.view(E4M3), s.k_scales.view(E8M0), s.v.view(E4M3), s.v_scales.view(E8M0))


def _finish(scores, v, seen, dtype):
    """Softmax over the last axis where `seen`, and its product with the values."""
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out.to(dtype), (top + torch.log(total)).squeeze(-1)


def _values(codes, scales):
    """Codes [..., D] and the bytes of their scales, as the numbers they stand for."""
    return codes.view(E4M3).float() * _two(scales.to(torch.int32) - 127)[..., None]


def _attend(s):
    c = s.case
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G, S, n = c["q_heads"] // H, c["seqs"], c["q_max"]
    L = s.cols * P
    starts, kv = s.q_starts.long(), s.kv_lens.long()
    j = torch.arange(L, device="cuda")
    filled = (j[None] < kv[:, None]).view(S, s.cols, P, 1, 1)
    page = s.table.long().clamp(min=0)
    k = torch.where(filled, _values(s.k[page], s.k_scales[page][:, :, None]), 0.0)
    v = torch.where(filled, _values(s.v[page], s.v_scales[page][:, :, None]), 0.0)
    k = k.reshape(S, L, H, D).permute(0, 2, 3, 1)
    v = v.reshape(S, L, H, D).permute(0, 2, 1, 3)
    i = torch.arange(n, device="cuda")
    at = (starts[:-1, None] + i).clamp(max=s.T - 1)
    pos = (kv - (starts[1:] - starts[:-1]))[:, None] + i
    q = s.q[at].float().view(S, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    scores = torch.matmul(q, k) * (1.0 / math.sqrt(D))
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(S, 1, n, G, L).reshape(S, 1, n * G, L)
    out, lse = _finish(scores, v, seen, s.q.dtype)
    seq, _ = _places(s)
    row = torch.arange(s.T, device="cuda") - starts[seq]
    out = out.view(S, H, n, G, D).permute(0, 2, 1, 3, 4)[seq, row].reshape(s.T, H * G, D)
    lse = lse.view(S, H, n, G).permute(0, 2, 1, 3)[seq, row].reshape(s.T, H * G)
    return out, lse


def _sparse(s):
    c = s.case
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G = c["q_heads"] // H
    seq, pos = _places(s)
    pages = s.pages.long()
    page = s.table.long()[seq[:, None, None], pages.clamp(min=0)].clamp(min=0)
    h = torch.arange(H, device="cuda")[None, :, None]
    key = pages[..., None] * P + torch.arange(P, device="cuda")
    seen = (pages[..., None] >= 0) & (key <= pos[:, None, None, None])
    k = _values(s.k[page, :, h], s.k_scales[page, h][..., None])
    v = _values(s.v[page, :, h], s.v_scales[page, h][..., None])
    k = torch.where(seen[..., None], k, 0.0).flatten(2, 3)
    v = torch.where(seen[..., None], v, 0.0).flatten(2, 3)
    q = s.q.float().view(s.T, H, G, D)
    scores = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    out, lse = _finish(scores, v, seen.flatten(2)[:, :, None], s.q.dtype)
    return out.view(s.T, H * G, D), lse.view(s.T, H * G)


def _bounds(s):
    c = s.case
    P = c["page"]
    kv = s.kv_lens.long()
    starts = s.q_starts.long()
    # the pages that the new tokens went into, over all that they hold now
    first = (kv - (starts[1:] - starts[:-1])) // P
    idx = first[:, None] + torch.arange((c["q_max"] - 1) // P + 2, device="cuda")
    idx = torch.minimum(idx, ((kv - 1) // P)[:, None])
    page = s.table.long().gather(1, idx)
    j = idx[..., None] * P + torch.arange(P, device="cuda")
    filled = (j < kv[:, None, None])[..., None, None]
    k = _values(s.k[page], s.k_scales[page][:, :, None])
    s.bounds[page, :, 0] = torch.where(filled, k, float("inf")).amin(2).to(s.bounds.dtype)
    s.bounds[page, :, 1] = torch.where(filled, k, float("-inf")).amax(2).to(s.bounds.dtype)
    return s.bounds


def _resize(s, target, q_starts=None):
    """Each sequence to its target length: pages of those that shrink go to the top of the
    list of free ones, the last first; those that grow take theirs from its top."""
    P = s.case["page"]
    j = torch.arange(s.cols, device="cuda")
    have, want = -(-s.kv_lens.long() // P), -(-target.long() // P)
    gone = (j >= want[:, None]) & (j < have[:, None])
    r = gone.flatten().cumsum(0).view_as(gone)  # of each page that goes, from 1 on
    n = s.n_free.long()
    free = torch.cat([s.free, s.free.new_zeros(1)])
    free[torch.where(gone, n + r[-1, -1] - r, s.n_pages)] = s.table
    n = n + r[-1, -1]
    come = (j >= have[:, None]) & (j < want[:, None])
    i = come.flatten().cumsum(0).view_as(come)
    s.table.copy_(torch.where(come, free[torch.where(come, n - i, 0)], s.table))
    s.free.copy_(free[:-1])
    s.n_free.copy_(n - i[-1, -1])
    if q_starts is not None:  # rows of the new tokens, and where each goes
        new = (target - s.kv_lens).clamp(min=0).long()
        q_starts[0] = 0
        q_starts[1:] = new.cumsum(0)
        t = torch.arange(s.T, device="cuda")
        seq = torch.searchsorted(q_starts.long(), t, right=True) - 1
        pos = s.kv_lens.long()[seq] + t - q_starts.long()[seq]
        s.slots.copy_(s.table[seq, pos // P].long() * P + pos % P)
    s.kv_lens.copy_(target)


def _resize_both(s):
    q_starts = torch.empty(s.case["seqs"] + 1, dtype=torch.int32, device="cuda")
    if s.case["ended"]:
        _resize(s, s.low)
        _resize(s, s.high, q_starts)
    else:
        _resize(s, s.high, q_starts)
        _resize(s, s.low)
    return s.table, s.kv_lens, q_starts, s.slots, s.free, s.n_free


def run(s):
    c = s.case
    op = c["op"]
    if op == "tables":
        if not own:
            return _resize_both(s)
        t = s.tables
        if c["ended"]:
            t.resize(s.low)
            batch, slots = t.resize(s.high, s.T, c["q_max"], slots=s.slots)
        else:
            batch, slots = t.resize(s.high, s.T, c["q_max"], slots=s.slots)
            t.resize(s.low)
        return t.page_table, t.kv_lens, batch.q_starts, slots, t.free_pages, t.n_free
    if not own:
        return (_append(s) if op == "append" else _bounds(s) if op == "bounds"
                else _sparse(s) if c["pick"] else _attend(s))
    if op == "append":
        q = s.cache.append(s.batch, s.k_new, s.v_new, q=s.q, q_norm=s.q_norm, k_norm=s.k_norm,
                           eps=EPS, cos_sin=s.cos_sin, pairs=c["pairs"])
        return _cache_of(s, q)
    if op == "bounds":
        s.cache.update_bounds(s.batch, s.bounds)
        return s.bounds
    if c["pick"]:
        return s.cache.attention(s.batch, s.q, pages=s.pages, lse=True)
    return s.cache.attention(s.batch, s.q, window=c["window"], lse=True)


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    """The outputs from the definitions, one sequence after another, in 64 bits."""
    if c["op"] == "tables":
        return None  # whole numbers
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    P, H, D, Hq = c["page"], c["kv_heads"], c["dim"], c["q_heads"]
    G = Hq // H
    ends, kv, table = s.q_starts.tolist(), s.kv_lens.tolist(), s.table.long()
    f = torch.float64
    decode = torch.arange(256, dtype=torch.uint8, device="cuda").view(E4M3).to(f)

    def power(e):  # of two, exactly; NaN for a scale that is
        return torch.where(e > 127, float("nan"), ((e.long() + 1023) << 52).view(f))

    def numbers(codes, scales, used, L):
        """A sequence's first L keys (or values) [L, H, D]."""
        x = decode[codes[used].long()] * power(scales[used].long() - 127)[:, None, :, None]
        return x.reshape(-1, H, D)[:L]

    if c["op"] == "bounds":
        out = s.bounds.to(f)
        for b in range(c["seqs"]):
            first = (kv[b] - (ends[b + 1] - ends[b])) // P
            used = table[b, first:-(-kv[b] // P)]
            x = numbers(s.k, s.k_scales, used, len(used) * P).view(-1, P, H, D)
            last = kv[b] - (-(-kv[b] // P) - 1) * P  # tokens of the last page
            x[-1, last:] = x[-1, 0]
            out[used, :, 0], out[used, :, 1] = x.amin(1), x.amax(1)
        return out
    if c["op"] == "append":
        qo = torch.empty((s.T, Hq, D), dtype=f, device="cuda")
        vo, ve = decode[s.v.long()], s.v_scales.long() - 127
        codes = decode[:127]  # the numbers that are not negative, ascending
        for b in range(c["seqs"]):
            lo, hi, L = ends[b], ends[b + 1], kv[b]
            pos = torch.arange(L - (hi - lo), L, device="cuda")
            y = s.q[lo:hi].to(f)
            if c["norm"]:
                y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * s.q_norm.to(f)
            r = c["rot"]
            if r:
                y = y.clone()
                cs = s.cos_sin[pos].to(f)
                i0 = slice(0, r, 2) if c["pairs"] else slice(0, r // 2)
                i1 = slice(1, r, 2) if c["pairs"] else slice(r // 2, r)
                z = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
                z = z * torch.complex(y[..., i0], y[..., i1])
                y[..., i0], y[..., i1] = z.real, z.imag
            qo[lo:hi] = y
            # values go as they are: their codes are exact numbers
            first = L - (hi - lo)
            for p in range(first // P, (L - 1) // P + 1):
                at, lo_t, hi_t = table[b, p], max(first, p * P), min(L, (p + 1) * P)
                new = s.v_new[lo + lo_t - first:lo + hi_t - first].to(f)
                m = new.abs().amax((0, 2))
                e = torch.ceil(torch.log2(m / 448)).clamp(LOW, HIGH).long()
                e = torch.where(m > 448 * power(e), e + 1, e)  # where the logarithm was off
                e = torch.where(m <= 448 * power(e - 1), e - 1, e).clamp(LOW, HIGH)
                old = None
                if lo_t > p * P:
                    e = torch.maximum(e, ve[at])
                    old = vo[at, :lo_t - p * P] * power(ve[at] - e)[None, :, None]
                x = new * power(-e)[None, :, None]
                if old is not None:
                    x = torch.cat([old, x])
                # the nearest code, of two as near the even one
                a = x.abs().clamp(max=448.0)
                i = torch.searchsorted(codes, a.contiguous()).clamp(1, 126)
                below, above = a - codes[i - 1], codes[i] - a
                down = (below < above) | ((below == above) & ((i - 1) % 2 == 0))
                near = torch.where(down, codes[i - 1], codes[i])
                vo[at, hi_t - p * P - len(x):hi_t - p * P] = torch.where(x < 0, -near, near)
                ve[at] = e
        # a key next to the border of two codes falls to either side: none of them is its value
        return qo, None, None, vo, power(ve)
    out = torch.zeros((s.T, Hq, D), dtype=f, device="cuda")
    lse = torch.full((s.T, Hq), float("-inf"), dtype=f, device="cuda")
    for b in range(c["seqs"]):
        lo, hi, L = ends[b], ends[b + 1], kv[b]
        pos = torch.arange(L - (hi - lo), L, device="cuda")
        used = table[b, :-(-L // P)]
        k, v = numbers(s.k, s.k_scales, used, L), numbers(s.v, s.v_scales, used, L)
        j = torch.arange(L, device="cuda")
        seen = (j <= pos[:, None])[None]
        if c["window"]:
            seen = seen & (pos[:, None] - j < c["window"])[None]
        if c["pick"]:
            pick = torch.zeros((hi - lo, H, s.cols + 1), dtype=torch.bool, device="cuda")
            pick.scatter_(2, torch.where(s.pages[lo:hi] < 0, s.cols, s.pages[lo:hi]).long(), True)
            seen = seen & pick[:, :, j // P].permute(1, 0, 2)
        for h in range(H):
            mask = seen[h if seen.shape[0] > 1 else 0][:, None]
            q = s.q[lo:hi, h * G:(h + 1) * G].to(f)
            x = (q @ k[:, h].T / math.sqrt(D)).masked_fill(~mask, float("-inf"))
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[lo:hi, h * G:(h + 1) * G] = torch.softmax(x, -1).nan_to_num(0.0) @ v[:, h]
    return out, lse
