"""What a call of the paged cache's C entry points enqueues, over launches and a
runtime that only record (tests/paged_calls_host.cpp)."""
import os
import shutil
import subprocess

import pytest

from lossless_invariant_bit_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild.nvcc()))), "include")


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    out = str(tmp_path_factory.mktemp("paged_calls") / "calls")
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CUDA, "-I", libbuild.INCLUDE, "-I",
                    libbuild.CSRC, os.path.join(HERE, "paged_calls_host.cpp"), "-x", "c++",
                    os.path.join(libbuild.CSRC, "ibp_paged_api.cu"), "-o", out],
                   check=True)
    return out


def test_calls_that_share_a_workspace_are_enqueued_whole(calls):
    r = subprocess.run([calls, "threads"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "whole"


def test_calls_with_a_workspace_each_do_not_wait_for_each_other(calls):
    r = subprocess.run([calls, "apart"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "mixed"
