"""The loop that takes a weight gradient's tiles over loses none, run on the host from the kernel's
header (CPU only)."""
import os
import subprocess

from mixture_experts_layer_65_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_tile_is_lost(tmp_path):
    exe = str(tmp_path / "host_tile_takeover")
    cmd = [build.nvcc_path(), "-gencode", build.GENCODE, "-O2", "-std=c++17",
           "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
           "-o", exe, os.path.join(HERE, "host_tile_takeover.cu")]
    comp = subprocess.run(cmd, capture_output=True, text=True)
    assert comp.returncode == 0, comp.stdout + comp.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "no tile is lost" in run.stdout
