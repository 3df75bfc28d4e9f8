"""The paged K/V cache at its edges, against plain 64-bit implementations with the
bounds of test_gpu_paged.py."""
import threading

import pytest
import torch

from lossless_invariant_bit_gb300 import paged
from tests.gpu_util import DEV
from tests.test_gpu_paged import Setup

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    """Calls of several threads share their stream's workspace; tiles here are cut, so
    their pieces go through it, in batches of one kernel, of the other, and of both."""
    sets = [Setup([300, 1, 1, 5], [3001, 4000, 77, 2000], G=8, D=128, dtype=torch.bfloat16, seed=1),
            Setup([1, 1], [9001, 3], G=4, H=3, D=64, seed=2),
            Setup([700, 1], [5000, 4999], G=7, D=128, dtype=torch.bfloat16, seed=3)]
    want = [st.cache.attention(st.batch, st.q, lse=True) for st in sets]
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(len(sets))

    def calls(i):
        st = sets[i]
        begin.wait()
        got = [st.cache.attention(st.batch, st.q, lse=True) for _ in range(150)]
        torch.cuda.current_stream().synchronize()
        wrong.extend(i for a in got if not (torch.equal(a[0], want[i][0])
                                            and torch.equal(a[1], want[i][1])))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert all(st.cache.status() == 0 for st in sets)


def test_stream_handle_zero_is_the_default_stream():
    assert paged._as_stream(0).cuda_stream == 0
    side = torch.cuda.Stream()
    assert paged._as_stream(side.cuda_stream).cuda_stream == side.cuda_stream
    assert paged._as_stream(side) is side
    st = Setup([1, 9], [40, 30], G=2, D=64)
    want = st.cache.attention(st.batch, st.q)
    assert torch.equal(st.cache.attention(st.batch, st.q, stream=0), want)


def test_empty_arguments_are_not_absent_ones():
    """A tensor without elements has a null pointer, which tells the library that it
    was not given: attention over no pages is not attention over every key."""
    st = Setup([2], [40], G=2, D=64, poison=False)
    k = torch.zeros((2, 2, 64), dtype=st.dtype, device=DEV)
    with pytest.raises(ValueError):
        st.cache.attention(st.batch, st.q, pages=torch.zeros((2, 2, 0), dtype=torch.int32,
                                                             device=DEV))
    for shape in ((0, 64), (64, 0)):
        with pytest.raises(ValueError):
            st.cache.append(st.batch, k, k, q=st.q, cos_sin=torch.zeros(shape, device=DEV))
    with pytest.raises(ValueError):
        st.cache.append(st.batch, k, k, q=st.q[:, :0])
