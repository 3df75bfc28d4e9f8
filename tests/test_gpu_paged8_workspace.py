"""What attention over 8-bit pages takes and leaves of the device's memory."""
import pytest
import torch

from lossless_invariant_bit_gb300 import ibp
from lossless_invariant_bit_gb300.paged import PagedCache
from tests.gpu_util import DEV
from tests.test_gpu_paged8 import BF16_WEIGHT, Setup, attend

pytestmark = pytest.mark.gpu


def test_the_larger_workspace_is_given_back():
    """A stream keeps the ordinary workspace, also where its calls took more."""
    s = Setup([1600], [1600], 1, 2, 128, 16, torch.bfloat16)
    table = torch.full((1, 6000), -1, dtype=torch.int32, device=DEV)
    table[:, :s.cols] = s.table
    s.table, s.batch = table, s.cache.batch(table, s.batch.kv_lens, s.batch.q_starts, s.T, 1600)
    more = ibp.ibp_paged_workspace(s.cache.handle, s.batch.desc, 2) - ibp.PAGED_WORKSPACE_BYTES
    assert more > 64 << 20
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = s.cache.attention(s.batch, s.q)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            with torch.cuda.stream(st):
                again = s.cache.attention(s.batch, s.q)
        torch.cuda.synchronize()
        assert torch.equal(again, out)
        del again
    held = torch.cuda.memory_allocated() - before
    assert held <= 3 * ibp.PAGED_WORKSPACE_BYTES + (1 << 20)
    s.check(*attend(s), weight=BF16_WEIGHT)


def test_weights_over_codes_whatever_memory_is_free():
    """most_workspace=0: weights are rounded to fp16, with room and without the same bits."""
    s = Setup([900], [3000], 2, 2, 128, 32, torch.bfloat16)
    s.check(*attend(s), weight=BF16_WEIGHT)
    s.cache.most_workspace = 0
    out, lse = attend(s)
    s.check(out, lse)
    c = PagedCache(2, 128, 32, s.n_pages, torch.bfloat16, k=s.cache.k, v=s.cache.v,
                   page_dtype=torch.float8_e4m3fn, k_scales=s.cache.k_scales,
                   v_scales=s.cache.v_scales, most_workspace=0)
    assert torch.equal(c.attention(s.batch, s.q), out) and c.status() == 0
