"""Products grouped by expert on the GPU against 64-bit products of the same inputs, element by
element (tolerances: tests/operators_ref.py)."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200._call import DTYPES
from mixture_experts_layer_65_b200._lib import lib
from mixture_experts_layer_65_b200.grouped import grouped_mm, grouped_mm_dgrad, grouped_mm_wgrad
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _inputs(op, counts, n, k, dt, tail=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = sum(counts) + tail
    x = torch.randn(rows, k, generator=g, device="cuda").to(dt)
    dy = torch.randn(rows, n, generator=g, device="cuda").to(dt)
    w = torch.randn(len(counts), n, k, generator=g, device="cuda").to(dt)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return {"mm": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[op] + (c,)


FN = {"mm": grouped_mm, "dgrad": grouped_mm_dgrad, "wgrad": grouped_mm_wgrad}


def _check(op, a, b, c, got, rows=None):
    ref, tol = R.grouped(op, a, b, c)
    got = got[:ref.shape[0]] if op != "wgrad" else got
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (op, int(bad.sum()), float((got.double() - ref).abs()[bad].max()))


# counts that end inside, at and behind every tile's border; experts without rows, one that has all
COUNTS = {
    "one_row": [1],
    "ones": [1, 0, 1, 1, 0, 0, 1],
    "borders": [15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129],
    "big": [0, 300, 0, 0, 513, 255, 1, 256, 0],
    "one_has_all": [0, 0, 700, 0],
    "few_each": [6, 3, 0, 9, 12, 5, 8, 7] * 4,
    "none": [0, 0, 0],
}
# widths inside and across the tiles
WIDTHS = [(8, 8), (64, 128), (136, 72), (264, 520), (320, 192), (33, 67), (256, 1)]


@pytest.mark.parametrize("n,k", WIDTHS, ids=lambda v: str(v))
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_products_match_64_bits(op, dt, counts, n, k):
    a, b, c = _inputs(op, counts, n, k, DT[dt], tail=5)
    got = FN[op](a, b, c)
    _check(op, a, b, c, got)
    torch.testing.assert_close(FN[op](a, b, c)[:sum(counts)] if op != "wgrad" else FN[op](a, b, c),
                               got[:sum(counts)] if op != "wgrad" else got, rtol=0, atol=0)


@pytest.mark.parametrize("op,n,k,counts", [
    ("mm", 2816, 2048, [9, 0, 5, 7, 6, 3, 1, 8]), ("mm", 1408, 2048, [700, 1, 300, 513]),
    ("dgrad", 1408, 2048, [10, 0, 129, 3]), ("dgrad", 896, 1280, [1000, 515, 0, 77]),
    ("wgrad", 1408, 2048, [515, 0, 1000, 3]), ("wgrad", 896, 1280, [5, 1, 17, 0, 30]),
], ids=lambda v: str(v) if not isinstance(v, list) else "c%d" % sum(v))
def test_products_at_layer_widths(op, n, k, counts):
    a, b, c = _inputs(op, counts, n, k, torch.bfloat16)
    _check(op, a, b, c, FN[op](a, b, c))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["mm", "dgrad"])
@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 200, 77]])
def test_rows_behind_the_last_expert_stay(op, dt, counts):
    n, k, tail = 136, 264, 70
    a, b, c = _inputs(op, counts, n, k, DT[dt], tail=tail)
    a[sum(counts):] = float("nan")
    out = torch.full((a.shape[0], n if op == "mm" else k), 7.0, dtype=DT[dt], device="cuda")
    got = FN[op](a, b, c, out=out)
    assert got is out
    assert bool((out[sum(counts):] == 7.0).all())
    _check(op, a[:sum(counts)], b, c, out[:sum(counts)])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_other_experts_rows_do_not_reach_a_result(dt):
    """NaN and infinity in one expert's rows (and behind the last) leave the others alone."""
    counts, n, k = [37, 5, 130, 64, 3], 136, 72
    for op in ("mm", "dgrad", "wgrad"):
        a, b, c = _inputs(op, counts, n, k, DT[dt], tail=9)
        clean = FN[op](a, b, c)
        lo, hi = 37, 42
        a[lo:hi] = float("nan")
        a[sum(counts):] = float("inf")
        if op == "wgrad":
            b[lo:hi] = float("inf")
            b[sum(counts):] = float("nan")
        got = FN[op](a, b, c)
        if op == "wgrad":
            keep = [0, 2, 3, 4]
            assert torch.equal(got[keep], clean[keep])
            assert bool(got[1].isnan().all())
        else:
            assert torch.equal(got[:lo], clean[:lo]) and torch.equal(got[hi:sum(counts)], clean[hi:sum(counts)])
            assert bool(got[lo:hi].isnan().all())


@pytest.mark.parametrize("counts", [[40, -7, 30, 0], [40, 50, 60, 70], [2**31 - 1, 5, 2**31 - 1, 3],
                                    [-1, -1, -2**31, 4]])
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("n,k", [(72, 136), (33, 35)])
def test_counts_that_do_not_fit_are_cut(op, counts, n, k):
    rows = 100
    a, b, _ = _inputs(op, [rows], n, k, torch.bfloat16)
    if op != "wgrad":
        b = torch.randn(len(counts), n, k, device="cuda").to(torch.bfloat16)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = None if op == "wgrad" else torch.full((rows, n if op == "mm" else k), 3.0, dtype=torch.bfloat16,
                                                device="cuda")
    got = FN[op](a, b, c, out=out)
    last = R.bounds(counts, rows)[-1]
    if op != "wgrad":
        assert bool((got[last:] == 3.0).all())
        got = got[:last]
    _check(op, a, b, c, got)


@pytest.mark.parametrize("dt,n,k", [("bf16", 136, 264), ("bf16", 35, 33), ("fp32", 40, 24)])
def test_weight_gradients_accumulate(dt, n, k):
    counts = [70, 0, 300, 1]
    dy, x, c = _inputs("wgrad", counts, n, k, DT[dt])
    base = torch.randn(len(counts), n, k, device="cuda")
    got = grouped_mm_wgrad(dy, x, c, out=base.clone(), accumulate=True)
    ref, tol = R.grouped("wgrad", dy, x, c)
    ref = ref + base.double()
    assert bool(((got.double() - ref).abs() <= tol + R.E * ref.abs() + 2 * R.E * tol).all())
    assert torch.equal(got[1], base[1])     # no rows: as it was
    assert torch.equal(grouped_mm_wgrad(dy, x, c, out=base.clone())[1], torch.zeros_like(base[1]))


# few tiles and many rows: the rows are split; parts that are empty, ragged, one expert with all
SPLIT = {"even": [9000, 9000], "ragged": [20001, 3, 0, 1], "one": [30011]}


@pytest.mark.parametrize("counts", SPLIT.values(), ids=SPLIT.keys())
@pytest.mark.parametrize("dt,n,k", [("bf16", 64, 136), ("bf16", 33, 35), ("fp32", 64, 40), ("fp32", 33, 35)])
def test_long_weight_gradients_are_split(dt, n, k, counts):
    dy, x, c = _inputs("wgrad", counts, n, k, DT[dt], tail=3)
    dy[sum(counts):] = float("nan")
    assert lib().moe_grouped_wgrad_workspace(len(counts), dy.shape[0], n, k, DTYPES[DT[dt]]) > 0
    got = grouped_mm_wgrad(dy, x, c)
    _check("wgrad", dy[:sum(counts)], x[:sum(counts)], c, got)
    assert torch.equal(grouped_mm_wgrad(dy, x, c), got)
    base = torch.randn(len(counts), n, k, device="cuda")
    acc = grouped_mm_wgrad(dy, x, c, out=base.clone(), accumulate=True)
    assert torch.equal(acc, base + got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = grouped_mm_wgrad(dy, x, c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, got)


@pytest.mark.parametrize("dt,n,k,q", [("bf16", 64, 64, 100000), ("fp32", 64, 64, 100000), ("bf16", 33, 67, 100000),
                                      ("fp32", 40, 64, 4096)])
def test_long_sums_keep_their_precision(dt, n, k, q):
    """The norm of the error over the norm of the result: below 1e-6, whatever the length of the
    sum (a single chain of 100,000 fp32 additions, or of truncating ones, is at 1e-5)."""
    if q == 4096:
        a, b, c = _inputs("mm", [300], n, q, DT[dt])
        got, ref = grouped_mm(a, b, c), R.grouped("mm", a, b, c)[0]
    else:
        a, b, c = _inputs("wgrad", [q], n, k, DT[dt])
        got, ref = grouped_mm_wgrad(a, b, c), R.grouped("wgrad", a, b, c)[0]
    assert float((got.double() - ref).norm() / ref.norm()) < 1e-6


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_unaligned_views_and_many_groups(op):
    counts = [(3 * i) % 5 for i in range(1024)]
    a, b, c = _inputs(op, counts, 16, 24, torch.bfloat16)
    _check(op, a, b, c, FN[op](a, b, c))
    shift = torch.empty(a.numel() + 1, dtype=a.dtype, device="cuda")[1:].view(a.shape).copy_(a)
    assert shift.data_ptr() % 16 != 0
    _check(op, shift, b, c, FN[op](shift, b, c))


# operands that start at any element, in memory whose other elements are NaN
@pytest.mark.parametrize("off_a,off_b", [(i, (3 * i + 1) % 8) for i in range(8)])
@pytest.mark.parametrize("n,k,counts", [(33, 35, [5, 0, 40, 1]), (77, 130, [129, 3, 64]), (700, 645, [900, 0, 531]),
                                        (1, 9, [3]), (64, 48, [70, 2])])
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_operands_that_start_anywhere(op, n, k, counts, off_a, off_b):
    a, b, c = _inputs(op, counts, n, k, torch.bfloat16, seed=off_a)

    def moved(t, off):
        room = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device="cuda")
        return room[8 + off:8 + off + t.numel()].view(t.shape).copy_(t)

    _check(op, a, b, c, FN[op](moved(a, off_a), moved(b, off_b), c))


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_no_rows_at_all(op):
    a, b, c = _inputs(op, [0, 0], 64, 72, torch.bfloat16)
    got = FN[op](a, b, c)
    assert got.numel() == 0 if op != "wgrad" else not got.any()


def test_gradients_agree_with_differences():
    """dgrad and wgrad against central differences of mm (fp32, a linear map: the only error is
    the products' own rounding over the step)."""
    counts, n, k, h = [5, 0, 9], 7, 6, 0.5
    x, w, c = _inputs("mm", counts, n, k, torch.float32)
    dy = torch.randn(sum(counts), n, device="cuda")
    dx, dw = grouped_mm_dgrad(dy, w, c), grouped_mm_wgrad(dy, x, c)

    def loss(x, w):
        return float((grouped_mm(x, w, c).double() * dy.double()).sum())

    for t, d, at in ((x, dx, [(0, 0), (4, 5), (13, 2)]), (w, dw, [(0, 3, 1), (1, 0, 0), (2, 6, 5)])):
        for i in at:
            p, m = t.clone(), t.clone()
            p[i] += h
            m[i] -= h
            a = [p if t is x else x, p if t is w else w]
            b = [m if t is x else x, m if t is w else w]
            num = (loss(*a) - loss(*b)) / (p[i] - m[i]).double().item()
            # each loss: 14 rows x 7 outputs of 6 products, 8 E of their magnitudes
            mag = float((grouped_mm(x.abs() + h, w.abs() + h, c).double() * dy.double().abs()).sum())
            assert abs(num - float(d[i])) <= 2 * 8 * R.E * mag / (2 * h) + 64 * R.E * mag


def test_another_stream_and_a_captured_graph():
    counts = [130, 0, 5, 64]
    res = {}
    args = {op: _inputs(op, counts, 136, 264, torch.bfloat16, seed=3) for op in FN}
    for op, (a, b, c) in args.items():
        res[op] = FN[op](a, b, c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for op, (a, b, c) in args.items():
        got = FN[op](a, b, c, stream=side)
        side.synchronize()
        assert torch.equal(got, res[op])
    outs = {op: torch.empty_like(r) for op, r in res.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op, (a, b, c) in args.items():
            FN[op](a, b, c, out=outs[op])
    for _ in range(2):
        for o in outs.values():
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for op in FN:
            assert torch.equal(outs[op], res[op])


def test_bindings_refuse():
    x, w, c = _inputs("mm", [4, 4], 16, 24, torch.bfloat16)
    with pytest.raises(ValueError, match="wide"):
        grouped_mm(x, torch.zeros(2, 16, 32, dtype=torch.bfloat16, device="cuda"), c)
    with pytest.raises(ValueError, match="counts"):
        grouped_mm(x, w, c.long())
    with pytest.raises(ValueError, match="counts"):
        grouped_mm(x, w, c.cpu())
    with pytest.raises(ValueError, match="w must"):
        grouped_mm(x, w.float(), c)
    with pytest.raises(ValueError, match="contiguous"):
        grouped_mm(x.t().contiguous().t(), w, c)
    with pytest.raises(ValueError, match="out"):
        grouped_mm(x, w, c, out=torch.empty(8, 15, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="give it"):
        grouped_mm_wgrad(x, x, c, accumulate=True)
    with pytest.raises(ValueError, match="float32"):
        grouped_mm_wgrad(x, x, c, out=torch.empty(2, 24, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(RuntimeError, match="overlaps"):
        grouped_mm(x, torch.zeros(2, 24, 24, dtype=torch.bfloat16, device="cuda"), c, out=x)
    with pytest.raises(ValueError, match="contiguous"):
        grouped_mm(x.half(), w.half(), c)
