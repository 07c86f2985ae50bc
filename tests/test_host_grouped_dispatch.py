"""The GPU tests' shapes reach every kernel of the grouped products: the rules, compiled from the
kernels' headers into a host program, say which one each shape takes (CPU only)."""
import os
import subprocess

from mixture_experts_layer_65_b200 import build
from tests.grouped_cases import CASES, TAIL

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_kernel_has_a_case(tmp_path):
    exe = str(tmp_path / "host_grouped_dispatch")
    cmd = [build.nvcc_path(), "-gencode", build.GENCODE, "-O2", "-std=c++17",
           "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
           "-o", exe, os.path.join(HERE, "host_grouped_dispatch.cu")]
    comp = subprocess.run(cmd, capture_output=True, text=True)
    assert comp.returncode == 0, comp.stdout + comp.stderr
    lines = [f"{op} {dt} {len(c)} {sum(c) + TAIL} {n} {k}" for op, dt, c, n, k, _ in CASES]
    run = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr
    assert list(zip(lines, run.stdout.splitlines())) == list(zip(lines, (c[-1] for c in CASES)))
    reached = {(op, kernel.split(" parts")[0]) for op, _, _, _, _, kernel in CASES}
    for op in ("mm", "dgrad", "wgrad"):
        assert {(op, f"simt {side} {v}") for side in (64, 128) for v in (1, 4)} <= reached
        assert {(op, "simt 32 1"), (op, "warp 64"), (op, "warp 128")} <= reached
        assert {(op, "tma")} <= reached if op == "wgrad" else {(op, "tma 64"), (op, "tma 256")} <= reached
    assert {"simt", "warp", "tma"} == {c[-1].split()[0] for c in CASES if "parts" in c[-1]}
