"""Host-side checks of the paged K/V cache that need no GPU."""
import ctypes

import pytest

from lossless_invariant_bit_gb300 import build as libbuild
from lossless_invariant_bit_gb300 import ibp


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ibp._lib_handle()


def desc(**kw):
    d = dict(k=4096, v=8192, page_stride=16 * 2 * 64 * 2, head_stride=128, token_stride=256,
             n_pages=4, page_tokens=16, kv_heads=2, head_dim=64, dtype=1)
    d.update(kw)
    return ibp.ibp_paged_desc(*[d[f] for f, _ in ibp.ibp_paged_desc._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), "IBP_EINVAL"), (dict(v=None), "IBP_EINVAL"), (dict(n_pages=0), "IBP_EINVAL"),
    (dict(page_tokens=4), "IBP_EINVAL"), (dict(page_tokens=24), "IBP_EINVAL"),
    (dict(page_tokens=512), "IBP_EINVAL"), (dict(head_dim=0), "IBP_EINVAL"),
    (dict(head_dim=72), "IBP_EINVAL"), (dict(head_dim=256), "IBP_EINVAL"),
    (dict(kv_heads=0), "IBP_EINVAL"), (dict(dtype=2), "IBP_EINVAL"),
    (dict(token_stride=64), "IBP_EINVAL"), (dict(head_stride=0), "IBP_EINVAL"),
    (dict(page_stride=1 << 41), "IBP_EINVAL"), (dict(k=4098), "IBP_EALIGN"),
    (dict(v=8200), "IBP_EALIGN"), (dict(token_stride=264), "IBP_EALIGN"),
])
def test_create_refuses(lib, kw, code):
    out = ctypes.c_void_p(1)
    d = desc(**kw)
    assert lib.ibp_paged_create(ctypes.byref(out), ctypes.addressof(d)) == getattr(ibp, code)
    assert out.value is None
    assert lib.ibp_paged_create(None, ctypes.addressof(d)) == ibp.IBP_EINVAL


def test_null_handles(lib):
    b = ibp.ibp_paged_batch()
    pb = ctypes.addressof(b)
    st = ctypes.c_int()
    assert lib.ibp_paged_create(ctypes.byref(ctypes.c_void_p()), None) == ibp.IBP_EINVAL
    assert lib.ibp_paged_destroy(None) == ibp.IBP_OK
    assert lib.ibp_paged_status(None, None, ctypes.byref(st), 0) == ibp.IBP_EINVAL
    assert lib.ibp_paged_append(None, pb, 16, 16, 256, None, 0, None, 0, 0, None, None, 1e-6, None,
                                0, 0, 0, None) == ibp.IBP_EINVAL
    assert lib.ibp_paged_attention(None, pb, 16, 256, 2, 16, None, 1.0, 1, 0, None, 0, 16, 1 << 30,
                                   None) == ibp.IBP_EINVAL
    assert lib.ibp_paged_bounds(None, pb, 16, None) == ibp.IBP_EINVAL
    assert lib.ibp_paged_scores(None, pb, 16, 256, 2, 16, 16, None) == ibp.IBP_EINVAL
    assert lib.ibp_paged_select(None, pb, 16, 1, 16, None) == ibp.IBP_EINVAL


def test_structures_match_the_header(lib):
    """The binding's structures and workspace size against the header's text."""
    import re

    text = open(ibp.HEADER).read()
    for name in ("ibp_paged_desc", "ibp_paged_batch"):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = re.findall(r"(void\*|const int32_t\*|uint64_t|uint32_t)\s+(\w+);", body)
        kinds = {"void*": ctypes.c_void_p, "const int32_t*": ctypes.c_void_p,
                 "uint64_t": ctypes.c_uint64, "uint32_t": ctypes.c_uint32}
        assert [(n, kinds[t]) for t, n in fields] == getattr(ibp, name)._fields_
    mib = int(re.search(r"IBP_PAGED_WORKSPACE_BYTES \((\d+)ull << 20\)", text).group(1))
    assert ibp.PAGED_WORKSPACE_BYTES == mib << 20
