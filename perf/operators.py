"""The operators of the paged K/V cache: cases, inputs, plain forms and 64-bit values.

The K/V cache of a model that is being served lives in pages: `page` tokens of
one sequence, `kv_heads` heads of `dim` 16-bit values each, found through a
page table.  Five operators work on it, each reached through `PagedCache`:

  append   a step's keys and values into their pages; keys (and queries) are
           normalised for each head and rotated by their position on the way
  attend   a ragged batch of new tokens (one of a sequence that is being
           answered, many of a prompt's chunk) over everything in its pages
  score    each page's bounds (the smallest and largest key of each channel),
           and for each query an upper bound of its products with a page's keys
  select   the pages with the largest scores of each query and K/V head
  sparse   attention over the selected pages alone

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _case(name, op, seqs, q_max, kv_max, q_heads, kv_heads, dim, page, dtype, lens=0, **more):
    c = {"op": op, "seqs": seqs, "q_max": q_max, "kv_max": kv_max, "q_heads": q_heads,
         "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "lens": lens,
         "layout": "rows"}
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token of each of the 20 sequences of the K/V workload (32 heads of 128, fp16)
        # goes into the cache, rotated, without norms: a decode step's append
        _case("append_step", "append", 20, 1, 1984, 32, 32, 128, 16, "fp16",
              norm=False, rot=128, pairs=False),
        # prompts of odd lengths, 64 query heads on 8 K/V heads, with the norms of each head:
        # the append of a prefill step
        _case("append_prompt", "append", 11, 1531, 4000, 64, 8, 128, 32, "bf16", lens=5,
              norm=True, rot=128, pairs=False),
        # one user, a short conversation: latency
        _case("attend_one", "attend", 1, 1, 517, 32, 32, 128, 16, "fp16", window=0),
        # the K/V workload's decode step: 20 sequences of 1920 + 64 tokens, 32 heads of 128
        _case("attend_step", "attend", 20, 1, 1984, 32, 32, 128, 16, "fp16", window=0),
        # a server's mixed batch: sequences that are being answered beside chunks of prompts,
        # odd lengths, heads of 64, a sliding window
        _case("attend_mixed", "attend", 24, 333, 6001, 32, 4, 64, 32, "bf16", lens=7,
              window=2500),
        # chunked prefill: 2048 new tokens behind 6144 cached ones, 64 query heads on 8
        _case("attend_chunk", "attend", 1, 2048, 8192, 64, 8, 128, 64, "bf16", window=0,
              layout="heads"),
        # 16 long sequences, one token each: the bounds of the newest page, every page's score
        _case("score_step", "score", 16, 1, 32768, 32, 8, 128, 16, "bf16"),
        # a small chunk behind a context of odd length
        _case("score_chunk", "score", 3, 61, 5003, 16, 4, 64, 32, "fp16", lens=3),
        # 128 of up to 2048 pages for each of 16 tokens and 8 K/V heads
        _case("select_step", "select", 16, 1, 32768, 32, 8, 128, 16, "bf16", pick=128),
        # a chunk's tokens, each with its own pages
        _case("select_chunk", "select", 2, 509, 16001, 32, 8, 128, 16, "bf16", lens=2, pick=33),
        # 16 long sequences, one token each, over 128 pages of 16 tokens out of up to 2048
        _case("sparse_step", "sparse", 16, 1, 32768, 32, 8, 128, 16, "bf16", pick=128, window=0),
        # tokens of a chunk, each over its own 24 pages of 32
        _case("sparse_chunk", "sparse", 2, 119, 4099, 32, 4, 128, 32, "fp16", lens=4, pick=24,
              window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("append", "attend", "attend", "score", "select", "sparse"))
        kv_heads = rng.choice((1, 2, 3, 4, 8, 8, 16, 32))
        group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
        seqs = _log(rng, 1, 64)
        q_max = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        kv_max = q_max + _log(rng, 1, 32768)
        c = _case(None, op, seqs, q_max, kv_max, kv_heads * group, kv_heads,
                  rng.choice((64, 80, 96, 128, 128)), rng.choice((8, 16, 16, 32, 64, 128)),
                  rng.choice(("bf16", "fp16")), lens=rng.randint(0, 999),
                  layout=rng.choice(("rows", "heads")))
        if c["q_heads"] > 128:
            continue
        if op == "append":
            c["norm"], c["pairs"] = rng.random() < 0.5, rng.random() < 0.5
            c["rot"] = rng.choice((0, c["dim"] // 32 * 16, c["dim"] // 16 * 16))
        if op in ("attend", "sparse"):
            c["window"] = 0 if op == "sparse" or rng.random() < 0.6 else _log(rng, 1, kv_max)
        if op in ("select", "sparse"):
            c["pick"] = _log(rng, 1, 256)
            if op == "select" and kv_max // c["page"] < 2 * c["pick"] + 6:
                continue  # nothing to choose from
        w = work(c)
        pool = sum(-(-n // c["page"]) for n in _lens(c)[1]) * c["page"] * kv_heads * c["dim"] * 4
        pages, tokens = -(-kv_max // c["page"]), sum(_lens(c)[0])
        plain = {"append": 0,
                 "attend": 4 * seqs * q_max * kv_max * c["q_heads"],
                 "score": 4 * seqs * q_max * pages * c["q_heads"],
                 "select": 4 * tokens * kv_heads * pages,
                 "sparse": 4 * tokens * kv_heads * c.get("pick", 0) * c["page"] * c["dim"]}[op]
        if w["flops"] > 4.4e11 or w["bytes"] > 1.2e9 or pool > 6e9 or plain > 1.2e10:
            continue
        return c


def _lens(c):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    if not c["lens"]:
        return [c["q_max"]] * c["seqs"], [c["kv_max"]] * c["seqs"]
    r = random.Random(c["lens"])
    q, kv = [], []
    for i in range(c["seqs"]):
        n = c["q_max"] if i == 0 else 1 if r.random() < 0.5 else r.randint(1, c["q_max"])
        q.append(n)
        kv.append(c["kv_max"] if i == 0 else r.randint(max(n, c["kv_max"] // 8), c["kv_max"]))
    return q, kv


def work(c):
    """Bytes that have to be read and written and operations that have to be done."""
    q, kv = _lens(c)
    T, D, H, P = sum(q), c["dim"], c["kv_heads"], c["page"]
    G = c["q_heads"] // H
    rows = 2 * T * D  # bytes of one head of every token
    if c["op"] == "append":
        n = 2 * rows * (c["q_heads"] + 2 * H) + 4 * T * c["rot"]
        return {"bytes": n, "flops": (4 * c["norm"] + 3 * bool(c["rot"])) * T * D * (c["q_heads"] + H)}
    pages = [-(-n // P) for n in kv]
    if c["op"] == "attend":
        win = c["window"] or 1 << 62
        pairs = keys = 0
        for n, l in zip(q, kv):
            first = l - n  # position of the first new token
            pairs += sum(min(first + i + 1, win) for i in range(n))
            keys += l - max(0, first + 1 - win)
        return {"bytes": 2 * rows * c["q_heads"] + 4 * T * c["q_heads"] + 4 * keys * H * D,
                "flops": 4 * D * c["q_heads"] * pairs}
    seen = sum(sum((l - n + i) // P + 1 for i in range(n)) for n, l in zip(q, kv))
    if c["op"] == "score":
        touched = sum((l - 1) // P - (l - n) // P + 1 for n, l in zip(q, kv))
        return {"bytes": rows * c["q_heads"] + 4 * sum(pages) * H * D
                + touched * H * D * (2 * P + 4) + 4 * T * H * max(pages),
                "flops": 4 * D * c["q_heads"] * seen}
    if c["op"] == "select":
        return {"bytes": 4 * H * seen + 4 * T * H * c["pick"], "flops": H * seen}
    keys = pairs = 0
    for n, l in zip(q, kv):
        own_pairs = [min((l - n + i) // P, c["pick"] - 1) * P + (l - n + i) % P + 1
                     for i in range(n)]
        pairs += sum(own_pairs)
        keys += min(l, sum(own_pairs))
    return {"bytes": 2 * rows * c["q_heads"] + 4 * T * c["q_heads"] + 4 * T * H * c["pick"]
            + 4 * keys * H * D, "flops": 4 * D * c["q_heads"] * pairs}


# ---------------------------------------------------------------- inputs
class State:
    pass


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(c, seed):
    s = State()
    s.case = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    q, kv = _lens(c)
    P, H, D = c["page"], c["kv_heads"], c["dim"]
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
    if c["op"] != "select":
        # keys with a scale of their own for each channel; memory that no token has been
        # written to holds what it may (NaN), but for the append, whose pages are returned
        shape = (n_pages, P, H, D) if c["layout"] == "rows" else (n_pages, H, P, D)
        chan = torch.exp(0.3 * _rand(g, H, D))
        s.k = torch.empty(shape, dtype=dt, device="cuda")
        s.v = torch.empty(shape, dtype=dt, device="cuda")
        if c["layout"] == "heads":
            s.k, s.v = s.k.transpose(1, 2), s.v.transpose(1, 2)
        s.k.copy_(s.k.new_empty(s.k.shape).normal_(generator=g) * chan.to(dt))
        s.v.copy_(s.v.new_empty(s.v.shape).normal_(generator=g))
        free = torch.ones(n_pages, dtype=torch.bool, device="cuda")
        free[s.table[live].long()] = False
        tail = torch.arange(P, device="cuda")[None] >= (s.kv_lens - 1)[:, None] % P + 1
        last = s.table.gather(1, (lens - 1)[:, None]).long()[:, 0]
        hole = free[:, None].repeat(1, P)
        hole[last] |= tail
        nothing = 0.0 if c["op"] == "append" else float("nan")
        s.k[hole] = nothing
        s.v[hole] = nothing
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
    elif c["op"] != "select":
        s.q = _rand(g, T, c["q_heads"], D).to(dt)
    if c["op"] == "score":
        s.bounds = torch.stack([s.k.nan_to_num(0.0).amin(1), s.k.nan_to_num(0.0).amax(1)], 2)
    if c["op"] in ("select", "sparse"):
        s.scores = _rand(g, T, H, cols)
        seq, pos = _places(s)
        hidden = torch.arange(cols, device="cuda")[None] > pos[:, None] // P
        s.scores.masked_fill_(hidden[:, None], float("-inf"))
    if c["op"] == "sparse":
        s.pages = _select(s, s.scores)
        del s.scores
    if own:
        from lossless_invariant_bit_gb300.paged import PagedCache

        if c["op"] == "select":
            s.cache = PagedCache(H, D, P, n_pages, dt)
        else:
            s.cache = PagedCache(H, D, P, n_pages, dt, k=s.k, v=s.v)
        s.batch = s.cache.batch(s.table, s.kv_lens, s.q_starts, T, c["q_max"])
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


def _append(s):
    c = s.case
    seq, pos = _places(s)
    cs = s.cos_sin[pos] if c["rot"] else None
    q = _rotate(_norm(s.q, s.q_norm), cs, c["rot"], c["pairs"]).to(s.q.dtype)
    k = _rotate(_norm(s.k_new, s.k_norm), cs, c["rot"], c["pairs"]).to(s.q.dtype)
    page, slot = s.table[seq, pos // c["page"]].long(), pos % c["page"]
    s.k[page, slot] = k
    s.v[page, slot] = s.v_new
    return q, s.k, s.v


def _finish(scores, v, seen, dtype):
    """Softmax over the last axis where `seen`, and its product with the values."""
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out.to(dtype), (top + torch.log(total)).squeeze(-1)


def _attend(s):
    c = s.case
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G, S, n = c["q_heads"] // H, c["seqs"], c["q_max"]
    L = s.cols * P
    starts, kv = s.q_starts.long(), s.kv_lens.long()
    j = torch.arange(L, device="cuda")
    filled = (j[None] < kv[:, None]).view(S, s.cols, P, 1, 1)
    page = s.table.long().clamp(min=0)
    k = torch.where(filled, s.k[page], 0.0).float().reshape(S, L, H, D).permute(0, 2, 3, 1)
    v = torch.where(filled, s.v[page], 0.0).float().reshape(S, L, H, D).permute(0, 2, 1, 3)
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
    seq, tpos = _places(s)
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
    k = torch.where(seen[..., None], s.k[page, :, h], 0.0).float().flatten(2, 3)
    v = torch.where(seen[..., None], s.v[page, :, h], 0.0).float().flatten(2, 3)
    q = s.q.float().view(s.T, H, G, D)
    scores = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    out, lse = _finish(scores, v, seen.flatten(2)[:, :, None], s.q.dtype)
    return out.view(s.T, H * G, D), lse.view(s.T, H * G)


def _score(s):
    c = s.case
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G, S, n = c["q_heads"] // H, c["seqs"], c["q_max"]
    starts, kv = s.q_starts.long(), s.kv_lens.long()
    count = starts[1:] - starts[:-1]
    # the pages that the new tokens went into, over all that they hold now
    first = (kv - count) // P
    idx = first[:, None] + torch.arange((n - 1) // P + 2, device="cuda")
    idx = torch.minimum(idx, ((kv - 1) // P)[:, None])
    page = s.table.long().gather(1, idx)
    j = idx[..., None] * P + torch.arange(P, device="cuda")
    filled = (j < kv[:, None, None])[..., None, None]
    k = s.k[page]
    s.bounds[page, :, 0] = torch.where(filled, k, float("inf")).amin(2)
    s.bounds[page, :, 1] = torch.where(filled, k, float("-inf")).amax(2)
    # sum over d of max(q lo, q hi) = sum of max(q, 0) hi + min(q, 0) lo
    b = s.bounds[s.table.long().clamp(min=0)].float()  # [S, pages, H, 2, D]
    at = (starts[:-1, None] + torch.arange(n, device="cuda")).clamp(max=s.T - 1)
    q = s.q[at].float().view(S, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    sc = torch.matmul(q.clamp(min=0), b[..., 1, :].permute(0, 2, 3, 1))
    sc += torch.matmul(q.clamp(max=0), b[..., 0, :].permute(0, 2, 3, 1))
    sc = sc.view(S, H, n, G, s.cols).amax(3).permute(0, 2, 1, 3)
    seq, pos = _places(s)
    sc = sc[seq, torch.arange(s.T, device="cuda") - starts[seq]]
    hidden = torch.arange(s.cols, device="cuda")[None] > pos[:, None] // P
    return s.bounds, torch.where(hidden[:, None], float("-inf"), sc)


def _select(s, scores):
    c = s.case
    seq, pos = _places(s)
    newest = (pos // c["page"])[:, None, None]
    j = torch.arange(s.cols, device="cuda")
    scores = torch.where(j == newest, float("inf"), scores)
    order = torch.sort(scores, dim=-1, descending=True, stable=True).indices[..., :c["pick"]]
    order = torch.where(order > newest, 1 << 30, order).sort(-1).values
    out = torch.where(order == 1 << 30, -1, order).to(torch.int32)
    missing = c["pick"] - out.shape[-1]
    return torch.cat([out, out.new_full((*out.shape[:-1], missing), -1)], -1)


def run(s):
    c = s.case
    op = c["op"]
    if not own:
        return _select(s, s.scores) if op == "select" else globals()["_" + op](s)
    if op == "append":
        q = s.cache.append(s.batch, s.k_new, s.v_new, q=s.q, q_norm=s.q_norm, k_norm=s.k_norm,
                           eps=EPS, cos_sin=s.cos_sin, pairs=c["pairs"])
        return q, s.k, s.v
    if op == "attend":
        return s.cache.attention(s.batch, s.q, window=c["window"], lse=True)
    if op == "sparse":
        return s.cache.attention(s.batch, s.q, pages=s.pages, lse=True)
    if op == "score":
        s.cache.update_bounds(s.batch, s.bounds)
        return s.bounds, s.cache.page_scores(s.batch, s.q, s.bounds)
    return s.cache.select_pages(s.batch, s.scores, c["pick"])


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    """The outputs from the definitions, one sequence after another, in 64 bits."""
    if c["op"] == "select":
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
    if c["op"] == "append":
        qo = torch.empty((s.T, Hq, D), dtype=f, device="cuda")
        ko, vo = s.k.to(f), s.v.to(f)
    out = torch.zeros((s.T, Hq, D), dtype=f, device="cuda")
    lse = torch.full((s.T, Hq), float("-inf"), dtype=f, device="cuda")
    if c["op"] == "score":
        bo = s.bounds.to(f)
        so = torch.full((s.T, H, s.cols), float("-inf"), dtype=f, device="cuda")
    for b in range(c["seqs"]):
        lo, hi, L = ends[b], ends[b + 1], kv[b]
        pos = torch.arange(L - (hi - lo), L, device="cuda")
        used = table[b, :-(-L // P)]
        if c["op"] == "append":
            for src, w, dst in ((s.q, s.q_norm, qo), (s.k_new, s.k_norm, ko)):
                x = src[lo:hi].to(f)
                if w is not None:
                    x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.to(f)
                r = c["rot"]
                y = x.clone()
                if r:
                    cs = s.cos_sin[pos].to(f)
                    z = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
                    i0 = slice(0, r, 2) if c["pairs"] else slice(0, r // 2)
                    i1 = slice(1, r, 2) if c["pairs"] else slice(r // 2, r)
                    z = z * torch.complex(x[..., i0], x[..., i1])
                    y[..., i0], y[..., i1] = z.real, z.imag
                if dst is qo:
                    qo[lo:hi] = y
                else:
                    ko[used[pos // P], pos % P] = y
            vo[used[pos // P], pos % P] = s.v_new[lo:hi].to(f)
            continue
        if c["op"] == "score":
            for p in range((L - (hi - lo)) // P, (L - 1) // P + 1):
                kp = s.k[used[p], :min(P, L - p * P)].to(f)
                bo[used[p], :, 0], bo[used[p], :, 1] = kp.amin(0), kp.amax(0)
            bb = bo[used]  # [pages, H, 2, D]
            for h in range(H):
                q = s.q[lo:hi, h * G:(h + 1) * G].to(f)
                mid = (bb[:, h, 0] + bb[:, h, 1]) / 2
                rad = (bb[:, h, 1] - bb[:, h, 0]) / 2
                so[lo:hi, h, :len(used)] = (q @ mid.T + q.abs() @ rad.T).amax(1)
            hidden = torch.arange(s.cols, device="cuda")[None] > pos[:, None] // P
            so[lo:hi].masked_fill_(hidden[:, None], float("-inf"))
            continue
        k = s.k[used].reshape(-1, H, D)[:L].to(f)
        v = s.v[used].reshape(-1, H, D)[:L].to(f)
        j = torch.arange(L, device="cuda")
        seen = (j <= pos[:, None])[None]
        if c["op"] == "attend" and c["window"]:
            seen = seen & (pos[:, None] - j < c["window"])[None]
        if c["op"] == "sparse":
            pick = torch.zeros((hi - lo, H, s.cols + 1), dtype=torch.bool, device="cuda")
            pick.scatter_(2, torch.where(s.pages[lo:hi] < 0, s.cols, s.pages[lo:hi]).long(), True)
            seen = seen & pick[:, :, j // P].permute(1, 0, 2)
        for h in range(H):
            mask = seen[h if seen.shape[0] > 1 else 0][:, None]
            q = s.q[lo:hi, h * G:(h + 1) * G].to(f)
            x = (q @ k[:, h].T / math.sqrt(D)).masked_fill(~mask, float("-inf"))
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[lo:hi, h * G:(h + 1) * G] = torch.softmax(x, -1).nan_to_num(0.0) @ v[:, h]
    if c["op"] == "append":
        return qo, ko, vo
    return (bo, so) if c["op"] == "score" else (out, lse)
