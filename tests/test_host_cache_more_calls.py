"""Host side of weights, evictions and reads on stand-ins for the CUDA runtime: host threads, refusals (no GPU)."""
import os
import subprocess

import pytest

from prefill_decode_paged_gb300 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cache") / "cache_more_host_check")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(kbuild.nvcc_path()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, "-I", cuda,
                    os.path.join(HERE, "csrc", "cache_more_host_check.cpp"), os.path.join(kbuild.CSRC, "cache.cpp"),
                    os.path.join(kbuild.CSRC, "cache_more.cpp"), "-o", exe], check=True)
    return exe


def play(harness, what):
    out = subprocess.run([harness, what], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout


def test_an_evictions_steps_stay_together_among_host_threads(harness):
    play(harness, "threads")


def test_an_empty_table_is_not_an_eviction_in_place(harness):
    play(harness, "into")


def test_rows_that_are_read_into_do_not_overlap(harness):
    play(harness, "overlap")
