"""In which order calls of several threads on page tables are enqueued, over a launch and a
runtime that only record (tests/paged_tables_host.cpp)."""
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
    out = str(tmp_path_factory.mktemp("paged_tables") / "calls")
    api = [os.path.join(libbuild.CSRC, f) for f in ("ibp_paged_api.cu", "ibp_paged8_api.cu")]
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CUDA, "-I", libbuild.INCLUDE, "-I",
                    libbuild.CSRC, os.path.join(HERE, "paged_tables_host.cpp"), "-x", "c++", *api,
                    "-o", out], check=True)
    return out


@pytest.mark.parametrize("how,want", [("threads", "whole"), ("apart", "mixed")])
def test_calls_on_the_same_tables_are_enqueued_whole(calls, how, want):
    r = subprocess.run([calls, how], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == want
