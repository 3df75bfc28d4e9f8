"""The workspace that attention over 8-bit pages is given, without a GPU."""
import ctypes

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp, paged
from tests.test_paged_binding_host import F16, I32, Library, Said, lib  # noqa: F401
from tests.test_paged8_host import E4M3, E8M0, made  # noqa: F401

BF16 = torch.bfloat16


class Asks(Library):
    """As Library, with room for 16-bit pages wanted; keeps what attention is given."""

    wants = ibp.PAGED_WORKSPACE_BYTES

    def ibp_paged_workspace(self, handle, batch, heads, out):
        self.called.append(("ibp_paged_workspace", heads))
        ctypes.cast(out, ctypes.POINTER(ctypes.c_uint64))[0] = self.wants
        return ibp.IBP_OK

    def ibp_paged_attention(self, *args):
        self.called.append(("ibp_paged_attention", args[-2]))
        return ibp.IBP_OK


@pytest.fixture
def asks(made, monkeypatch):  # noqa: F811
    fake = Asks()
    monkeypatch.setattr(ibp, "_lib_handle", lambda: fake)
    monkeypatch.setattr(paged, "_large_workspace", lambda *a: Said((16,), torch.uint8))
    return fake


def attend(T, H, G, D, dtype, page_dtype=E4M3, pages=None, **more):
    shape = (5, 16, H, D)
    c = paged.PagedCache(H, D, 16, 5, dtype, k=Said(shape, page_dtype), v=Said(shape, page_dtype),
                         page_dtype=page_dtype,
                         **(dict(k_scales=Said((5, H), E8M0), v_scales=Said((5, H), E8M0))
                            if page_dtype is E4M3 else {}), **more)
    b = paged.PagedBatch(Said((1, 4), I32), Said((1,), I32), Said((2,), I32), T, T)
    q = Said((T, H * G, D), dtype)
    c.attention(b, q, out=q, pages=pages)


@pytest.mark.parametrize("T,H,G", [(64, 1, 128), (24, 1, 64), (1, 2, 1536), (17, 4, 1), (2048, 8, 8)])
def test_the_library_says_what_a_batch_makes_use_of(asks, T, H, G):
    """Also of few tokens with many queries each."""
    asks.wants = ibp.PAGED_WORKSPACE_BYTES + 4096
    attend(T, H, G, 128, BF16)
    assert asks.called == [("ibp_paged_workspace", H * G), ("ibp_paged_attention", asks.wants)]


def test_what_never_makes_use_of_more_does_not_ask(asks, monkeypatch):
    monkeypatch.setattr(ibp, "ibp_paged_create", lambda desc: 1)
    for kw in (dict(dtype=F16), dict(dtype=BF16, page_dtype=BF16),
               dict(dtype=BF16, pages=Said((100, 2, 3), I32))):
        attend(100, 2, 8, 128, **kw)
    attend(1, 2, 16, 128, BF16)
    attend(16, 8, 1, 128, BF16)
    assert asks.called == [("ibp_paged_attention", ibp.PAGED_WORKSPACE_BYTES)] * 5


def test_more_than_the_most_is_not_taken(asks):
    asks.wants = paged._MOST_WORKSPACE + 1
    attend(2048, 2, 8, 128, BF16)
    assert asks.called[1] == ("ibp_paged_attention", ibp.PAGED_WORKSPACE_BYTES)


def test_the_user_says_how_much_it_may_be(asks):
    """0: always the codes, with the rounding of their weights."""
    asks.wants = ibp.PAGED_WORKSPACE_BYTES + 4096
    for most, given in ((0, ibp.PAGED_WORKSPACE_BYTES), (asks.wants - 1, ibp.PAGED_WORKSPACE_BYTES),
                        (asks.wants, asks.wants), (None, asks.wants)):
        asks.called.clear()
        attend(2048, 2, 8, 128, BF16, most_workspace=most)
        assert asks.called[1] == ("ibp_paged_attention", given)
    with pytest.raises(ValueError):
        attend(2048, 2, 8, 128, BF16, most_workspace=-1)
