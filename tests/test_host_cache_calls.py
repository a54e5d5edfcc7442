"""The decode cache's host code on stand-ins for the CUDA runtime: host threads, devices."""
import os
import subprocess

import pytest

from prefill_decode_paged_gb300 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cache") / "cache_host_check")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(kbuild.nvcc_path()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, "-I", cuda,
                    os.path.join(HERE, "csrc", "cache_host_check.cpp"), "-o", exe], check=True)
    return exe


def play(harness, what):
    out = subprocess.run([harness, what], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout


def test_calls_of_host_threads_do_not_mix(harness):
    play(harness, "threads")


def test_status_is_of_the_caches_device(harness):
    play(harness, "device")
