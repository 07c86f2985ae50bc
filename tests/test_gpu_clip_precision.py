"""Clipped gradients are rounded once: max_norm, the norm and their quotient are 64-bit, and 48 bits
of the quotient meet the gradient.  So a result is off by half a step of fp32 (2^-24 of the value; the
coefficient's 2^-48 and the 64-bit sums' 1e-13 within the 0.1% allowed on top), bf16 ones by half of
their step more."""
import math

import pytest
import torch

from mixture_experts_layer_65_b200 import build, clip
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# limits that fp32 does not have: 0.9, 0.4 and 0.99 of its half step off
@pytest.mark.parametrize("limit", [1 + 0.9 * 2.0 ** -24, 1 - 0.4 * 2.0 ** -24, 3 + 0.99 * 2.0 ** -23, 0.7, 1e-3])
@pytest.mark.parametrize("dt", [F32, BF])
def test_scaled_gradients_are_rounded_once(dt, limit):
    gen = torch.Generator(device="cuda").manual_seed(0)
    before = [torch.randn(n, generator=gen, device="cuda").to(dt) for n in (5000, 33, 1)]
    norm = math.sqrt(R.norm_sq(before))

    def check(got):
        for g, b in zip(got, before):
            ref = b.double() * (limit / norm)
            tol = 1.001 * R.E + (R.half(BF) if dt == BF else 0)
            assert bool(((g.double() - ref).abs() <= tol * ref.abs()).all())

    got = [b.clone() for b in before]
    clip.clip_grad_norm(got, limit)
    check(got)
    outs = [torch.empty_like(b) for b in before]
    clip.scale_grads(before, torch.tensor([norm * norm], dtype=torch.float64, device="cuda"), limit, out=outs)
    check(outs)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("std,limit", [(1e37, 1e-3), (1e37, 1e-12), (1e30, 1e-5), (3e36, 1e-35), (1e12, 1e-19)])
def test_coefficients_below_the_fp32_range(dt, std, limit):
    """A norm of 10^39 and more is 64-bit; so is its quotient, down to 10^-75."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    before = [(torch.randn(n, generator=gen, device="cuda") * std).to(dt) for n in (5000, 33)]
    norm = math.sqrt(R.norm_sq(before))
    assert all(bool(b.isfinite().all()) for b in before)
    got = [b.clone() for b in before]
    clip.clip_grad_norm(got, limit)
    least = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps   # a step below the normal range
    for g, b in zip(got, before):
        ref = b.double() * (limit / norm)
        tol = 1.001 * R.E + (R.half(BF) if dt == BF else 0)
        assert bool(((g.double() - ref).abs() <= tol * ref.abs() + least).all())
    big = torch.cat([g.abs().double() for g in got]).max()
    assert float(big) > 0.01 * limit    # ordinary values come out of it
