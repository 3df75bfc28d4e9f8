"""When attention over 8-bit pages makes 16-bit ones, and what it enqueues, over launches and a
runtime that only record (tests/paged_stage_host.cpp)."""
import os
import shutil
import subprocess

import pytest

from lossless_invariant_bit_gb300 import build as libbuild
from tests.test_paged_calls_host import CUDA, HERE


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    out = str(tmp_path_factory.mktemp("paged_stage") / "calls")
    api = [os.path.join(libbuild.CSRC, f) for f in ("ibp_paged_api.cu", "ibp_paged8_api.cu")]
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CUDA, "-I", libbuild.INCLUDE, "-I",
                    libbuild.CSRC, os.path.join(HERE, "paged_stage_host.cpp"), "-x", "c++", *api,
                    "-o", out], check=True)
    return out


def run(calls, *args):
    r = subprocess.run([calls, *map(str, args)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    more, _, launches = r.stdout.strip().partition(" ")
    return int(more), launches


def room(H, D, pages):
    """A table for each (sequence, head), in whole kB; keys and values in 16 bits."""
    return -(-pages * H * 4 // 1024) * 1024 + 2 * pages * 16 * H * D * 2


ON_CODES = {1: "chunk8 join8", 2: "chunk8 behind8 join8"}
MADE = {1: "stage chunk16 join16", 2: "stage chunk16 behind8 join16"}


@pytest.mark.parametrize("D,H,Hq,seqs,cols,tokens,most", [
    (128, 8, 64, 1, 512, 192, 192),    # 6 tiles of 256 rows to a head, just
    (80, 1, 64, 1, 7, 24, 24),
    (128, 2, 4, 2, 100, 1536, 1000),   # 6 on the average of two
    (96, 4, 4, 1, 96, 1536, 1536),
])
def test_long_chunks_of_bf16(calls, D, H, Hq, seqs, cols, tokens, most):
    want = room(H, D, seqs * cols)
    args = (D, H, Hq, seqs, cols, tokens, most)
    kind = min(seqs, 2)
    assert run(calls, 1, *args, -1) == (want, MADE[kind])
    assert run(calls, 1, *args, want + 4096) == (want, MADE[kind])
    assert run(calls, 1, *args, -2) == (want, ON_CODES[kind])  # a byte too few
    assert run(calls, 1, *args, 0) == (want, ON_CODES[kind])
    assert run(calls, 0, *args, 1 << 30) == (0, ON_CODES[kind])  # fp16
    fewer = (D, H, Hq, seqs, cols, tokens - 1, most)
    assert run(calls, 1, *fewer, 1 << 30) == (0, ON_CODES[kind])


def test_heads_of_64_and_few_rows(calls):
    assert run(calls, 1, 64, 8, 64, 1, 512, 2048, 2048, 1 << 30) == (0, ON_CODES[1])
    assert run(calls, 1, 128, 8, 8, 1, 512, 16, 16, 1 << 30) == (0, "step8")
    # many sequences of which none may have more than 16 rows
    assert run(calls, 1, 128, 1, 16, 4, 512, 9000, 1, 1 << 30) == (0, "step8")
