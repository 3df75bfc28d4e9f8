"""The 8-bit paged cache in a pool whose offsets pass 32 bits: the same calls as in a small
one give the same bits."""
import pytest
import torch

from lossless_invariant_bit_gb300.paged import PagedCache
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_pages_beyond_32_bits(dtype, layout):
    H, G, D, P = 8, 4, 128, 16
    q_lens, kv_lens = [1, 700, 1, 3], [900, 1000, 16, 300]
    need = [-(-n // P) for n in kv_lens]
    few, many = sum(need), (1 << 32) // (P * H * D) + 2 * sum(need)
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    perm = torch.randperm(few, generator=torch.Generator().manual_seed(0)).to(torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    table = table.to(DEV)
    starts = torch.tensor([0, 1, 701, 702, 705], dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    before = lens - (starts[1:] - starts[:-1])
    T, old = 705, int(before.sum())
    x = [torch.randn((old, h, D), generator=g, device=DEV).to(dtype) for h in (H, H)]
    k, v, q = (torch.randn((T, h, D), generator=g, device=DEV).to(dtype) for h in (H, H, H * G))
    results = []
    for n_pages in (few, many):
        shape = (n_pages, P, H, D) if layout == "rows" else (n_pages, H, P, D)
        codes = [torch.empty(shape, dtype=torch.uint8, device=DEV) for _ in range(2)]
        if layout == "heads":
            codes = [c.transpose(1, 2) for c in codes]
        scales = [torch.empty((n_pages, H), dtype=torch.uint8, device=DEV) for _ in range(2)]
        shift = n_pages - few  # the last pages
        assert shift == 0 or (shift * P * H * D) >> 32
        for c, s in zip(codes, scales):
            c[shift:], s[shift:] = 0, 0
        c = PagedCache(H, D, P, n_pages, dtype, k=codes[0].view(E4M3), v=codes[1].view(E4M3),
                       page_dtype=E4M3, k_scales=scales[0].view(torch.float8_e8m0fnu),
                       v_scales=scales[1].view(torch.float8_e8m0fnu))
        tab = torch.where(table >= 0, table + shift, table)
        first = torch.cat([before.new_zeros(1), before.cumsum(0).to(torch.int32)])
        c.append(c.batch(tab, before, first, old, int(before.max())), *x)
        b = c.batch(tab, lens, starts, T, 700)
        qo = c.append(b, k, v, q=q)
        bounds = torch.zeros((n_pages, H, 2, D), dtype=dtype, device=DEV)
        c.update_bounds(b, bounds)
        pages = c.select_pages(b, c.page_scores(b, qo, bounds), 5)
        outs = [*c.attention(b, qo, lse=True), c.attention(b, qo, pages=pages), pages]
        if dtype == torch.bfloat16:
            c.most_workspace = 0
            outs.append(c.attention(b, qo))
        one = c.batch(tab[:1], lens[:1], starts[:2], 1, 1)
        outs.append(c.attention(one, qo[:1]))
        assert c.status() == 0
        results.append([*outs, bounds[shift:].clone(), *(y[shift:].clone() for y in codes + scales)])
        del c, codes, scales, bounds, outs, b, one
        torch.cuda.empty_cache()
    for a, b in zip(*results):
        assert torch.equal(a, b)
