"""The attention kernels' division of keys among blocks, walked on the CPU."""
import os
import subprocess

from prefill_decode_paged_gb300 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_unit_has_one_part_and_every_join_finds_its_parts(tmp_path):
    exe = str(tmp_path / "cut_check")
    subprocess.run([kbuild.nvcc_path(), "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, os.path.join(HERE, "csrc", "cut_check.cu"),
                    "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout
