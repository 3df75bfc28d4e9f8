"""PagedCache's checks of its arguments, without a GPU: tensors that only say what
they are, and a library that counts its calls."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch

from lossless_invariant_bit_gb300 import ibp, paged


class Said:
    """What PagedCache asks of a tensor."""

    def __init__(self, shape, dtype, index=0):
        real = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self._real = real.shape, dtype, real
        self.index = index
        self.is_cuda = index >= 0
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def stride(self, i=None):
        return self._real.stride() if i is None else self._real.stride(i)

    def dim(self):
        return self._real.dim()

    def numel(self):
        return self._real.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Library:
    """Every entry point is called with success."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            return ibp.IBP_OK

        return call


T, H, G, D, P, N = 3, 2, 2, 64, 16, 5
F16, I32, F32 = torch.float16, torch.int32, torch.float32


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(ibp, "_lib_handle", lambda: fake)
    monkeypatch.setattr(ibp, "ibp_paged_create", lambda desc: 1)
    monkeypatch.setattr(ibp, "ibp_paged_destroy", lambda h: None)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(paged, "_workspace", lambda device, raw: Said((16,), torch.uint8))
    return fake


def a_cache(k=0, v=0):
    pages = (N, P, H, D)
    return paged.PagedCache(H, D, P, N, F16, k=Said(pages, F16, k), v=Said(pages, F16, v))


def a_batch(table=0, lens=0, starts=0):
    return paged.PagedBatch(Said((1, 4), I32, table), Said((1,), I32, lens),
                            Said((2,), I32, starts), T, T)


def arguments(**index):
    """Every call's tensors, on device 0 but those that `index` names."""
    kinds = dict(batch=None, k=((T, H, D), F16), v=((T, H, D), F16), q=((T, H * G, D), F16),
                 q_out=((T, H * G, D), F16), q_norm=((D,), F16), k_norm=((D,), F16),
                 cos_sin=((64, D), F32), out=((T, H * G, D), F16), pages=((T, H, 2), I32),
                 bounds=((N, H, 2, D), F16), scores=((T, H, 4), F32), scores_out=((T, H, 4), F32),
                 select_out=((T, H, 2), I32))
    out = {}
    for name, kind in kinds.items():
        i = index.get(name, 0)
        out[name] = a_batch(i, i, i) if kind is None else Said(*kind, i)
    return out


CALLS = {
    "ibp_paged_append": (lambda c, a: c.append(a["batch"], a["k"], a["v"], q=a["q"],
                                               q_norm=a["q_norm"], k_norm=a["k_norm"],
                                               cos_sin=a["cos_sin"], q_out=a["q_out"]),
                         ["batch", "k", "v", "q", "q_norm", "k_norm", "cos_sin", "q_out"]),
    "ibp_paged_attention": (lambda c, a: c.attention(a["batch"], a["q"], pages=a["pages"],
                                                     out=a["out"]),
                            ["batch", "q", "pages", "out"]),
    "ibp_paged_bounds": (lambda c, a: c.update_bounds(a["batch"], a["bounds"]),
                         ["batch", "bounds"]),
    "ibp_paged_scores": (lambda c, a: c.page_scores(a["batch"], a["q"], a["bounds"],
                                                    out=a["scores_out"]),
                         ["batch", "q", "bounds", "scores_out"]),
    "ibp_paged_select": (lambda c, a: c.select_pages(a["batch"], a["scores"], 2,
                                                     out=a["select_out"]),
                         ["batch", "scores", "select_out"]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_calls_take_what_is_on_the_caches_device(lib, name):
    call, _ = CALLS[name]
    call(a_cache(), arguments())
    assert lib.called == [name]


@pytest.mark.parametrize("name,which", [(n, w) for n in sorted(CALLS) for w in CALLS[n][1]])
@pytest.mark.parametrize("index", [-1, 1])
def test_calls_refuse_what_is_elsewhere(lib, name, which, index):
    """Host memory (-1) and another GPU's: nothing reaches the library."""
    call, _ = CALLS[name]
    with pytest.raises(ValueError):
        call(a_cache(), arguments(**{which: index}))
    assert not lib.called


def test_the_handle_is_made_on_the_pages_device(lib, monkeypatch):
    current, made = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ibp, "ibp_paged_create", lambda desc: made.append(current[-1]) or 1)
    a_cache(k=1, v=1)
    a_cache()
    assert made == [1, 0] and current == [0]


@pytest.mark.parametrize("kw", [dict(table=1), dict(lens=1), dict(starts=1), dict(table=-1)])
def test_a_batch_is_on_one_device(lib, kw):
    with pytest.raises(ValueError):
        a_batch(**kw)


@pytest.mark.parametrize("kw", [dict(k=1), dict(v=1), dict(k=-1, v=-1)])
def test_pages_are_on_one_device(lib, kw):
    with pytest.raises(ValueError):
        a_cache(**kw)


def test_the_module_loads_where_torch_has_no_cuda():
    """(A torch that was built without CUDA has no such function.)"""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from lossless_invariant_bit_gb300 import paged\n"
            "try:\n"
            "    paged.PagedCache(2, 64, 16, 4, torch.float32)\n"
            "except ValueError:\n"
            "    print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(paged.__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
