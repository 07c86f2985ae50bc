"""The block norms' parameter gradients are column sums over the rows.  A term has two to four
roundings, a CTA adds up its rows (one or two here) in fp32, the CTAs' sums meet in 64 bits and are
rounded once.  With independent errors of 0.41 E each (E = 2^-24), the norm of the error is that of a
sum of N random terms' errors, sqrt(5) * 0.41 E of the sum's norm, and 0.41 E for the last rounding:
1.1 E; 1.6 E are allowed."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200.block import block_norm, block_norm_backward
from tests import operators_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("T,d", [(1001, 333), (590, 1024), (1100, 2048)])
@pytest.mark.parametrize("post", [False, True])
def test_column_sums_meet_in_64_bits(T, d, post):
    g = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, y, dr, du, gate, wp = rnd(T, d), rnd(T, d), rnd(T, d), rnd(T, d), rnd(d), rnd(d)
    wq = rnd(d) if post else None
    fwd = block_norm(x, y, gate=gate, post_weight=wq, pre_weight=wp, beta=1.5)
    got = block_norm_backward(fwd, y, dr=dr, du=du, gate=gate, post_weight=wq, pre_weight=wp, beta=1.5)
    ref = R.norm_bwd(fwd, y, dr, du, gate, wq, wp, 1.5)
    pairs = [("d_gate", got.d_gate), ("d_pre", got.d_pre_weight)] + ([("d_post", got.d_post_weight)] if post else [])
    for name, t in pairs:
        v = ref[name][0]
        assert float((t.double() - v).norm() / v.norm()) <= 1.6 * R.E, name
