"""Backward of the block norms where the block's output holds infinities or NaN: without a norm after
the block, dy = g * gate has no y in it (tolerances: tests/operators_ref.py)."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200.block import block_norm, block_norm_backward
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 100), ("bf16", 512), ("bf16", 1280), ("bf16", 2001),
                                  ("bf16", 2056), ("bf16", 5000), ("bf16", 16384), ("fp32", 33), ("fp32", 333),
                                  ("fp32", 4096), ("fp32", 16384)])
def test_dy_does_not_read_y_without_a_norm_after_the_block(dt, d, gate, pre):
    T = 20
    g = torch.Generator(device="cuda").manual_seed(d)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, y, dr = rnd(T, d).to(DT[dt]), rnd(T, d).to(DT[dt]), rnd(T, d).to(DT[dt])
    gt = {"none": None, "channel": rnd(d), "token": rnd(T, 1)}[gate]
    wp, du = (rnd(d), rnd(T, d).to(DT[dt])) if pre else (None, None)
    fwd = block_norm(x, y, gate=gt, pre_weight=wp, beta=1.5)
    clean = block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, pre_weight=wp, beta=1.5)
    ref = R.norm_bwd(fwd, y, dr, du, gt, None, wp, 1.5)
    for got, name in ((clean.dx, "dx"), (clean.dy, "dy")):
        v, m = ref[name]
        tol = R.BWD * m + R.half(DT[dt]) * (v.abs() + R.BWD * m)
        assert bool(((got.double() - v).abs() <= tol).all())
    for row, value in ((1, float("inf")), (7, float("-inf")), (13, float("nan")), (19, float("inf"))):
        y[row, (row * 37) % d] = value
    y[3] = float("nan")
    got = block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, pre_weight=wp, beta=1.5)
    assert torch.equal(got.dx, clean.dx) and torch.equal(got.dy, clean.dy)
