"""Attention over 8-bit pages where scales and queries differ most: what the header says
is lost is lost, and nothing else."""
import math

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp, paged
from tests.gpu_util import DEV
from tests.test_gpu_paged8 import BF16_WEIGHT, E4M3, F64, Setup, attend

pytestmark = pytest.mark.gpu


def code_of(x):
    return int(torch.tensor(x).to(E4M3).view(torch.uint8))


# ---------------------------------------------------------------- values' scales in a block
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("spread", [11, 12, 22])
@pytest.mark.parametrize("n,L,window", [(40, 700, 0), (150, 700, 0), (200, 600, 300)])
def test_a_large_scale_beside_the_heaviest_key(n, L, window, spread, dtype):
    """The heaviest key (values of zero) shares its block with a page whose values' scale is
    2^spread larger, which a row does not see or gives no weight to; the result is
    the other keys', with weights of 2^-14 of the heaviest's.  (As many sequences and heads as
    give a CTA a tile's blocks one after the other.)"""
    s = Setup([n] * 30, [L] * 30, 2, 8, 64, 16, dtype, spread=0)
    k, v = s.codes
    heavy, large = 127, 6  # a position, a page: both of the first block
    pages = s.table.long()
    k[pages], v[pages] = 0, code_of(448.0)
    for sc in s.scales:
        sc[pages] = 127
    k[pages[:, heavy // 16], heavy % 16, :, 0] = code_of(1.0)
    v[pages[:, heavy // 16], heavy % 16] = 0
    k[pages[:, large], :, :, 1] = code_of(256.0)
    s.scales[1][pages[:, large]] = 127 + spread
    s.q.zero_()
    s.q[..., 0] = 14 * math.log(2.0)
    s.q[..., 1] = -1.0
    out, lse = attend(s, window=window, scale=1.0)
    s.check(out, lse, window=window, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_sums_of_many_equal_weights(dtype):
    """Every second page's keys have scales 2^-24 of the others', and scores of about zero: 10000
    equal weights, in blocks that take each page's scales.  (As many sequences and heads as
    give a CTA a hundred blocks of a tile.)"""
    s = Setup([130] * 10, [20000] * 10, 2, 8, 64, 16, dtype, spread=0)
    pages = s.table.long()
    s.scales[0][pages[:, ::2]] = 127 - 14
    s.scales[0][pages[:, 1::2]] = 127 + 10
    s.q *= 2.0 ** -17
    s.check(*attend(s))


# ---------------------------------------------------------------- factors of the scores
@pytest.mark.parametrize("n,L,wide", [(1, 200, False), (3, 200, True), (60, 300, False),
                                      (60, 300, True), (300, 500, False), (300, 500, True)])
def test_the_largest_queries_and_keys_of_zero(n, L, wide):
    """Queries near 2^120 under keys' scales of 2^50: scores of zero stay zero."""
    s = Setup([n], [L], 2, 2, 64, 16, torch.bfloat16, spread=0)
    pages = s.table[0].long()
    s.codes[0][pages] = 0
    s.scales[0][pages] = 177
    if wide:  # pages of one block that differ by more than a block's scale holds
        s.scales[0][pages[::2]] = 77
    s.q = (s.q.float() * 2.0 ** 120).bfloat16()
    s.check(*attend(s))


# ---------------------------------------------------------------- queries' range
def a_query_of_two_channels(n, L, small, keys):
    """q = (1, small) in two channels, keys zero in the first, `keys` x 1 to 4 in the second."""
    s = Setup([n], [L], 4, 2, 128, 16, torch.bfloat16, spread=0)
    pages = s.table[0].long()
    s.codes[0][pages] = 0
    few = torch.tensor([code_of(x) for x in (1.0, 1.5, 2.0, 3.0, 4.0)], dtype=torch.uint8,
                       device=DEV)
    pick = torch.randint(0, 5, s.codes[0][pages][..., 1].shape, generator=s.g, device=DEV)
    x = s.codes[0][pages]
    x[..., 1] = few[pick]
    s.codes[0][pages] = x
    s.scales[0][pages] = 127 + keys
    s.q.zero_()
    s.q[..., 0] = 1.0
    s.q[..., 1] = small
    return s


def scores_of(s):
    """Row 0's of the last token, and what the header allows each to be off by on codes."""
    K, _ = s.of(0, 0)
    q = s.q[-1, 0].to(F64)
    x = K[:, 0] @ q
    return x, 2.0 ** -39 * float(q.abs().max()) * K[:, 0].abs().sum(1)


@pytest.mark.parametrize("small,keys", [(2.0 ** -33 * 1.2421875, 32), (2.0 ** -40, 40)])
@pytest.mark.parametrize("n,L", [(1, 300), (4, 300), (500, 900)])
def test_a_query_with_one_large_channel(n, L, small, keys, monkeypatch):
    """A channel far below the row's largest that alone meets keys: over codes each score is off
    by 2^-39 max |q| sum |k| at most, over pages made 16-bit ones it is exact."""
    s = a_query_of_two_channels(n, L, small, keys)
    x, off = scores_of(s)
    want = float(torch.logsumexp(x, 0))
    room = ibp.ibp_paged_workspace(s.cache.handle, s.batch.desc, 8) > ibp.PAGED_WORKSPACE_BYTES
    assert room == (n == 500)
    if room:
        _, lse = attend(s, scale=1.0)
        assert abs(float(lse[-1, 0]) - want) <= 2.0 ** -18
        monkeypatch.setattr(paged, "_MOST_WORKSPACE", 0)
    _, lse = attend(s, scale=1.0)
    # the log of the sum moves by no more than the largest score does
    assert abs(float(lse[-1, 0]) - want) <= float(off.max()) + 2.0 ** -18
    assert s.cache.status() == 0


# ---------------------------------------------------------------- 16-bit pages of all scales
@pytest.mark.parametrize("q_lens,kv_lens,G,P", [([900], [1300], 2, 16), ([500, 700], [900, 1000], 4, 64)])
def test_long_chunks_of_bf16_under_scales_of_the_whole_range(q_lens, kv_lens, G, P):
    s = Setup(q_lens, kv_lens, G, 2, 128, P, torch.bfloat16, spread=0)
    for w, spread in ((0, 12), (1, 49)):
        live = s.scales[w] != 255
        x = torch.randint(127 - spread, 127 + spread + 1, s.scales[w].shape, generator=s.g,
                          device=DEV).to(torch.uint8)
        s.scales[w].copy_(torch.where(live, x, s.scales[w]))
    s.q *= 2.0 ** -8
    assert ibp.ibp_paged_workspace(s.cache.handle, s.batch.desc, 2 * G) > ibp.PAGED_WORKSPACE_BYTES
    s.check(*attend(s), weight=BF16_WEIGHT)
