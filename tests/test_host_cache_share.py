"""Which entries the threads of an eviction take, by the kernels' own header, on the CPU."""
import os
import subprocess

from prefill_decode_paged_gb300 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_shares_of_the_largest_evictions_against_64_bits(tmp_path):
    exe = str(tmp_path / "share_check")
    subprocess.run([kbuild.nvcc_path(), "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, os.path.join(HERE, "csrc", "share_check.cu"),
                    "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout
