"""Host-side checks of the 8-bit paged cache and the page tables that need no GPU."""
import ctypes
import re

import pytest
import torch

from lossless_invariant_bit_gb300 import build as libbuild
from lossless_invariant_bit_gb300 import ibp, paged
from tests.test_paged_binding_host import F16, I32, Said, lib  # noqa: F401
from tests.test_paged_host import desc

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def real():
    libbuild.build()
    return ibp._lib_handle()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), "IBP_EINVAL"), (dict(v=None), "IBP_EINVAL"), (dict(n_pages=0), "IBP_EINVAL"),
    (dict(page_tokens=4), "IBP_EINVAL"), (dict(page_tokens=24), "IBP_EINVAL"),
    (dict(head_dim=72), "IBP_EINVAL"), (dict(head_dim=144), "IBP_EINVAL"),
    (dict(dtype=2), "IBP_EINVAL"), (dict(token_stride=48), "IBP_EINVAL"),
    (dict(head_stride=48), "IBP_EINVAL"), (dict(k=4104), "IBP_EALIGN"),
    (dict(token_stride=136), "IBP_EALIGN"), (dict(head_stride=72), "IBP_EALIGN"),
    (dict(page_stride=1 << 41), "IBP_EINVAL"),
])
def test_create_refuses(real, kw, code):
    out = ctypes.c_void_p(1)
    d = desc(**dict(dict(page_stride=16 * 128, head_stride=64, token_stride=128), **kw))
    assert real.ibp_paged_create_8bit(ctypes.byref(out), ctypes.addressof(d), 16,
                                      32) == getattr(ibp, code)
    assert out.value is None


def test_null_arguments(real):
    d, t = desc(page_stride=2048, head_stride=64, token_stride=128), ibp.ibp_paged_tables()
    out = ctypes.c_void_p(1)
    assert real.ibp_paged_create_8bit(None, ctypes.addressof(d), 16, 16) == ibp.IBP_EINVAL
    assert real.ibp_paged_create_8bit(ctypes.byref(out), None, 16, 16) == ibp.IBP_EINVAL
    for ks, vs in ((None, 16), (16, None)):
        assert real.ibp_paged_create_8bit(ctypes.byref(out), ctypes.addressof(d), ks,
                                          vs) == ibp.IBP_EINVAL
        assert out.value is None
    n = ctypes.c_uint64(7)
    b = ibp.ibp_paged_batch()
    assert real.ibp_paged_workspace(None, ctypes.addressof(b), 8,
                                    ctypes.byref(n)) == ibp.IBP_EINVAL and n.value == 7
    assert real.ibp_paged_resize(None, ctypes.addressof(t), 16, 16, 16, 1, None) == ibp.IBP_EINVAL


def test_structure_matches_the_header():
    text = open(ibp.HEADER).read()
    body = re.search(r"typedef struct \{([^}]*)\} ibp_paged_tables;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"(int32_t\*|uint64_t|uint32_t)\s+(\w+);", body)
    kinds = {"int32_t*": ctypes.c_void_p, "uint64_t": ctypes.c_uint64, "uint32_t": ctypes.c_uint32}
    assert [(n, kinds[t]) for t, n in fields] == ibp.ibp_paged_tables._fields_


# ---------------------------------------------------------------- the binding's arguments
T, H, D, P, N = 3, 2, 64, 16, 5


def a_cache(**kw):
    pages, scales = (N, P, H, D), (N, H)
    a = dict(dtype=F16, k=Said(pages, E4M3), v=Said(pages, E4M3), page_dtype=E4M3,
             k_scales=Said(scales, E8M0), v_scales=Said(scales, E8M0))
    a.update(kw)
    return paged.PagedCache(H, D, P, N, **a)


@pytest.fixture
def made(lib, monkeypatch):  # noqa: F811
    log = []
    monkeypatch.setattr(ibp, "ibp_paged_create_8bit",
                        lambda d, ks, vs: log.append((d.token_stride, d.head_stride)) or 1)
    lib.made = log
    return lib


def test_a_cache_of_codes(made):
    c = a_cache()
    assert made.made == [(H * D, D)] and c.page_dtype is E4M3 and c.dtype is F16


@pytest.mark.parametrize("kw", [
    dict(page_dtype=torch.float8_e5m2), dict(page_dtype=torch.int8), dict(page_dtype=None),
    dict(k_scales=None), dict(v_scales=None), dict(k_scales=None, v_scales=None),
    dict(k=None, v=None), dict(k=Said((N, P, H, D), F16)), dict(v=Said((N, P, H, D), F16)),
    dict(k_scales=Said((N, H), torch.uint8)), dict(v_scales=Said((N, H + 1), E8M0)),
    dict(k_scales=Said((N, H), E8M0, 1)), dict(v_scales=Said((N, H), E8M0, -1)),
    dict(dtype=torch.float32), dict(dtype=E4M3),
])
def test_a_cache_refuses(made, kw):
    with pytest.raises(ValueError):
        a_cache(**kw)
    assert not made.made


def test_calls_take_the_16_bit_type(made):
    c = a_cache()
    b = paged.PagedBatch(Said((1, 4), I32), Said((1,), I32), Said((2,), I32), T, T)
    c.append(b, Said((T, H, D), F16), Said((T, H, D), F16))
    c.attention(b, Said((T, H, D), F16), out=Said((T, H, D), F16))
    assert made.called == ["ibp_paged_append", "ibp_paged_attention"]
    with pytest.raises(ValueError):
        c.append(b, Said((T, H, D), E4M3), Said((T, H, D), E4M3))
    with pytest.raises(ValueError):
        c.update_bounds(b, Said((N, H, 2, D), E4M3))


class Tables:
    """PageTables without their tensors."""

    def __new__(cls, cache):
        t = object.__new__(paged.PageTables)
        t.cache, t.n_seqs, t.max_pages = cache, 2, 4
        t.page_table, t.kv_lens = Said((2, 4), I32), Said((2,), I32)
        t.q_starts = Said((3,), I32)
        t._address, t._batches = 0, {}
        return t


@pytest.mark.parametrize("target,n,kw", [
    (Said((3,), I32), 0, {}), (Said((2,), torch.int64), 0, {}), (Said((2,), I32, 1), 0, {}),
    (Said((2,), I32, -1), 0, {}), (Said((2,), I32), -1, {}),
    (Said((2,), I32), 0, dict(slots=Said((0,), torch.int64))),
    (Said((2,), I32), 3, dict(slots=Said((2,), torch.int64))),
    (Said((2,), I32), 3, dict(slots=Said((3,), I32))),
    (Said((2,), I32), 3, dict(slots=Said((3,), torch.int64, 1))),
])
def test_resize_refuses(made, target, n, kw):
    with pytest.raises(ValueError):
        Tables(a_cache()).resize(target, n, **kw)
    assert not made.called


def test_a_shrinking_call_has_no_batch(made):
    assert Tables(a_cache()).resize(Said((2,), I32)) is None
    assert made.called == ["ibp_paged_resize"]


@pytest.mark.parametrize("n_seqs,max_pages", [(0, 4), (3, 0), (-1, 1)])
def test_tables_have_sequences_and_columns(made, n_seqs, max_pages):
    with pytest.raises(ValueError):
        a_cache().tables(n_seqs, max_pages)
