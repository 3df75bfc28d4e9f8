"""A decode loop over a paged K/V cache: prompts in chunks, then tokens one by one,
over every cached token or over the pages that score best; a sequence that pauses
leaves its pages for a compressed host store and comes back.

    python examples/paged_decode.py            # prints tokens per second of each form

The model here is one attention layer with random projections: what matters is
the order of the calls.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lossless_invariant_bit_gb300.paged import PagedCache  # noqa: E402
from lossless_invariant_bit_gb300.store import IbpStore  # noqa: E402


class Layer:
    """Projections of one attention layer, its norms and its rotation table."""

    def __init__(self, hidden, q_heads, kv_heads, dim, positions, dtype, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.wqkv = (rand((q_heads + 2 * kv_heads) * dim, hidden) / hidden ** 0.5).to(dtype)
        self.wo = (rand(hidden, q_heads * dim) / (q_heads * dim) ** 0.5).to(dtype)
        self.q_norm = torch.ones(dim, dtype=dtype, device="cuda")
        self.k_norm = torch.ones(dim, dtype=dtype, device="cuda")
        half = dim // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()

    def step(self, cache, batch, x, bounds=None, pick=0):
        """x [n_tokens, hidden] of the batch's new tokens -> the layer's output."""
        qkv = (x @ self.wqkv.T).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        q = cache.append(batch, k, v, q=q, q_norm=self.q_norm, k_norm=self.k_norm,
                         cos_sin=self.cos_sin)
        pages = None
        if bounds is not None:
            cache.update_bounds(batch, bounds)
            if pick:
                pages = cache.select_pages(batch, cache.page_scores(batch, q, bounds), pick)
        out = cache.attention(batch, q, pages=pages)
        return out.flatten(1) @ self.wo.T


def run(seqs=4, prompt=2000, chunk=512, steps=32, hidden=1024, q_heads=32, kv_heads=8, dim=128,
        page=16, pick=48, dtype=torch.bfloat16, seed=0):
    """Returns (outputs of the steps over every token, over the selected pages, the
    store's ratio of compressed to raw bytes, whether the paused sequence came back bit for
    bit, tokens per second of both forms)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    total = prompt + 2 * steps
    per = -(-total // page)
    layer = Layer(hidden, q_heads, kv_heads, dim, total, dtype, seed)
    cache = PagedCache(kv_heads, dim, page, (seqs + 1) * per, dtype)
    perm = torch.randperm((seqs + 1) * per, generator=g, device="cuda").to(torch.int32)
    table, spare = perm[:seqs * per].view(seqs, per).clone(), perm[seqs * per:]
    bounds = torch.zeros((cache.n_pages, kv_heads, 2, dim), dtype=dtype, device="cuda")

    def batch_of(lens, new):
        starts = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * new
        return cache.batch(table, torch.full((seqs,), lens, dtype=torch.int32, device="cuda"),
                           starts, seqs * new, new)

    x = torch.randn((seqs, total, hidden), generator=g, device="cuda").to(dtype)
    for at in range(0, prompt, chunk):  # prompts, a chunk of every sequence at a time
        n = min(chunk, prompt - at)
        layer.step(cache, batch_of(at + n, n), x[:, at:at + n].reshape(-1, hidden), bounds)

    def decode(first, pick):
        batch = batch_of(first, 1)  # its lengths grow in place
        outs = []
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(steps):
            batch.kv_lens.add_(1)
            outs.append(layer.step(cache, batch, x[:, first + i], bounds, pick))
        torch.cuda.synchronize()
        return torch.stack(outs), seqs * steps / (time.perf_counter() - t)

    full, full_rate = decode(prompt, 0)

    # sequence 0 pauses: a token's keys (values) are one row of the store
    rows = kv_heads * dim * 2
    held = prompt + steps
    at = torch.arange(held, device="cuda")
    old = table[0, at // page].long() * page + at % page
    table[0] = spare
    new = table[0, at // page].long() * page + at % page
    stored, same = 0, True
    for data in (cache.key_rows(), cache.value_rows()):
        seq = data[old].contiguous()
        store = IbpStore(rows, dim * 2, held)  # a chunk is one head
        try:
            store.build(seq)
            slots, sizes = store.compress(seq)  # pinned host memory
            stored += int(sizes.sum())
            data[old] = 0
            data[new] = store.gather(slots, at)  # and back, into other pages
            same = same and torch.equal(data[new], seq) and store.status() == 0
        finally:
            store.close()
    moved = torch.arange(-(-held // page), device="cuda")
    bounds[spare[moved].long()] = bounds[old[moved * page] // page]

    few, few_rate = decode(prompt + steps, pick)
    assert cache.status() == 0
    cache.close()
    return full, few, stored / (2 * held * rows), same, (full_rate, few_rate)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--seqs", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=16000)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--pick", type=int, default=64)
    a = ap.parse_args()
    run(seqs=2, prompt=600, steps=4)  # warm-up
    _, _, ratio, same, rates = run(a.seqs, a.prompt, steps=a.steps, pick=a.pick)
    print("%d sequences of %d tokens: %.0f tokens/s over every token, %.0f over %d pages of 16; "
          "a paused sequence stored at %.3f of its size, back bit for bit: %s"
          % (a.seqs, a.prompt, rates[0], rates[1], a.pick, ratio, same))


if __name__ == "__main__":
    main()
