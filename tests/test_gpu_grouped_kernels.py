"""Each kernel of the grouped products over several steps and pieces of its sums, against 64-bit
products of the same inputs (tests/grouped_cases.py has the shapes and says which kernel each takes).

Beside the bound by element (tests/operators_ref.py) a fp32 result is held to a norm of the error
below 1e-6 of the result's: a chain of c additions of random terms is off by about E sqrt(c / 6) of the
sum's norm, 7 E with 256 terms and 9 E with 480, so 17 E leaves out no product unseen."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200.grouped import device_status, grouped_mm, grouped_mm_dgrad, grouped_mm_wgrad
from tests import operators_ref as R
from tests.grouped_cases import CASES, TAIL

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FN = {"mm": grouped_mm, "dgrad": grouped_mm_dgrad, "wgrad": grouped_mm_wgrad}


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _inputs(op, counts, n, k, dt):
    """Rows behind the last expert's are NaN."""
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = sum(counts)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    def behind(t):
        return torch.cat([t, torch.full((TAIL, t.shape[1]), float("nan"), dtype=dt, device="cuda")])

    a = behind(rnd(rows, k if op == "mm" else n))
    b = behind(rnd(rows, k)) if op == "wgrad" else rnd(len(counts), n, k)
    return a, b, torch.tensor(counts, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("op,dt,counts,n,k,kernel", CASES,
                         ids=[f"{op}-{kernel.replace(' ', '_')}-{n}x{k}" for op, _, _, n, k, kernel in CASES])
def test_each_kernel_over_several_steps(op, dt, counts, n, k, kernel):
    a, b, c = _inputs(op, counts, n, k, DT[dt])
    rows = sum(counts)
    out = None
    if op != "wgrad":
        out = torch.full((rows + TAIL, n if op == "mm" else k), 7.0, dtype=DT[dt], device="cuda")
    got = FN[op](a, b, c, out=out)
    if op != "wgrad":
        assert bool((got[rows:] == 7.0).all())
        got = got[:rows]
    ref, tol = R.grouped(op, a[:rows], b[:rows] if op == "wgrad" else b, c)
    assert bool(((got.double() - ref).abs() <= tol).all())
    if got.dtype == torch.float32:
        for e, r in zip(got, ref) if op == "wgrad" else [(got, ref)]:
            assert float((e.double() - r).norm()) <= 1e-6 * float(r.norm())
    device_status()


def test_every_row_counts_past_31_bits_of_elements():
    """A weight gradient over a million rows, in 64-bit pieces."""
    n, k, tail = 64, 2048, 300
    rows = (1 << 31) // k + 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    c = torch.tensor([rows - tail, tail], dtype=torch.int32, device="cuda")
    dw = grouped_mm_wgrad(dy, x, c)
    ref = torch.zeros(2, n, k, dtype=torch.float64, device="cuda")
    for lo in range(0, rows - tail, 1 << 16):
        hi = min(rows - tail, lo + (1 << 16))
        ref[0] += dy[lo:hi].double().t() @ x[lo:hi].double()
    ref[1] = dy[rows - tail:].double().t() @ x[rows - tail:].double()
    # (one lost row of 1e6 would be 1e-3 of the norm)
    for got, want in zip(dw, ref):
        assert float((got.double() - want).norm()) <= 1e-6 * float(want.norm())
    device_status()
