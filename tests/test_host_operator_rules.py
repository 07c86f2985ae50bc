"""The grouped products' host-side rules (rings and tables inside shared memory, rows per tile,
splits of a weight gradient's rows), swept by a small host-only program compiled with nvcc from
the kernels' headers (CPU only: it makes no CUDA call)."""
import os
import subprocess

from mixture_experts_layer_65_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_operator_rules_hold(tmp_path):
    exe = str(tmp_path / "host_operator_rules")
    cmd = [build.nvcc_path(), "-gencode", build.GENCODE, "-O2", "-std=c++17",
           "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
           "-o", exe, os.path.join(HERE, "host_operator_rules.cu")]
    comp = subprocess.run(cmd, capture_output=True, text=True)
    assert comp.returncode == 0, comp.stdout + comp.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "all operator rules hold" in run.stdout
