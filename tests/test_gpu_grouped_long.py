"""bf16 mm and dgrad with long contractions: the tensor cores truncate when they add to an accumulator,
so chains are cut after 16,384 values.  Tolerance: half a bf16 step of the result, and per MMA step of
16 values of a chain two steps of fp32 (2^-23 each) of the terms' magnitudes: 1024 * 2^-22, with
the pieces' sums (at most 64 roundings) on top.  All terms are of one sign in half of the cases:
truncation then goes one way."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200.grouped import device_status, grouped_mm, grouped_mm_dgrad
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CHAIN = 1024 * 2.0 ** -22 + 64 * R.E


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# one chain, the first length that is cut, pieces that end inside a stage, many pieces; each width's
# kernel, in tiles of few and of many rows
@pytest.mark.parametrize("counts,other,length", [
    ([300, 0, 37], 520, 16384), ([300, 0, 37], 520, 16392), ([300, 0, 37], 264, 32832), ([5, 0, 30], 72, 16400),
    ([5, 0, 30], 72, 65600), ([37], 72, 1 << 18), ([37], 72, 1 << 20), ([700, 3], 72, 50000),
    ([300, 0, 37], 521, 16384), ([300, 0, 37], 521, 16385), ([5, 0, 30], 33, 40001), ([37], 65, (1 << 18) + 1),
    ([37], 9, (1 << 20) - 1), ([1300, 900, 200], 1027, 17001),
])
@pytest.mark.parametrize("op", ["mm", "dgrad"])
@pytest.mark.parametrize("positive", [False, True])
def test_long_contractions_keep_their_precision(op, counts, other, length, positive):
    g = torch.Generator(device="cuda").manual_seed(length)

    def rnd(*s):
        t = torch.randn(*s, generator=g, device="cuda")
        return (t.abs() if positive else t).to(BF)

    rows, G, tail = sum(counts), len(counts), 3
    a = torch.cat([rnd(rows, length), torch.full((tail, length), float("nan"), dtype=BF, device="cuda")])
    w = rnd(G, other, length) if op == "mm" else rnd(G, length, other)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full((rows + tail, other), 7.0, dtype=BF, device="cuda")
    (grouped_mm if op == "mm" else grouped_mm_dgrad)(a, w, c, out=out)
    again = (grouped_mm if op == "mm" else grouped_mm_dgrad)(a, w, c)
    assert bool((out[rows:] == 7.0).all()) and torch.equal(out[:rows], again[:rows])
    at = 0
    for e, n in enumerate(counts):
        x, m = a[at:at + n].double(), w[e].double().t() if op == "mm" else w[e].double()
        ref, t = x @ m, CHAIN * (x.abs() @ m.abs())
        assert bool(((out[at:at + n].double() - ref).abs() <= t + R.half(BF) * (ref.abs() + t)).all())
        at += n
    device_status()
