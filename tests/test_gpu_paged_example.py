"""The decode loop of examples/paged_decode.py, as a user runs it."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("paged_decode",
                                                  os.path.join(ROOT, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decode_loop():
    m = load()
    a = m.run(seqs=3, prompt=700, chunk=256, steps=6, hidden=256, q_heads=8, kv_heads=2, dim=64,
              pick=1000)
    full, few, ratio, same, _ = a
    assert same and 0 < ratio <= 1.0
    for x in (full, few):
        assert x.shape == (6, 3, 256) and bool(torch.isfinite(x.float()).all())
    # with every page selected the second decode is plain attention over the pages that came
    # back: the loop run again with no selection gives it, but for the order of the sums
    b = m.run(seqs=3, prompt=700, chunk=256, steps=6, hidden=256, q_heads=8, kv_heads=2, dim=64,
              pick=0)
    assert torch.equal(full, b[0])
    d = (few.double() - b[1].double()).norm() / b[1].double().norm()
    assert d < 2.0 ** -7  # two roundings to bf16 on either side of a projection
