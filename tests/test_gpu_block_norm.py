"""The norms around a block on the GPU against the 64-bit formulas, element by element
(tolerances: tests/operators_ref.py)."""
import itertools

import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200.block import BlockNorm, block_norm, block_norm_backward
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _inputs(T, d, dt, gate, post, pre, seed=0, with_y=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, y = (2 * rnd(T, d)).to(dt), rnd(T, d).to(dt)
    gt = {"none": None, "channel": rnd(d), "token": rnd(T, 1)}[gate]
    wq, wp = rnd(d) if post else None, rnd(d) if pre else None
    dr, du = rnd(T, d).to(dt), rnd(T, d).to(dt) if pre else None
    return x, y if with_y else None, gt, wq, wp, dr, du


def _close(name, got, ref, tol):
    if ref is None:
        assert got is None, name
        return
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(((got.double() - ref).abs() / tol)[bad].max()))


def _check_fwd(x, y, gt, wq, wp, beta, got):
    r, u, sy, sr, _ = R.norm_fwd(x, y, gt, wq, wp, beta, EPS)
    tr, tu, ty, ts = R.norm_fwd_tol(x, y, gt, wq, wp, beta, EPS, x.dtype)
    if y is None:
        assert got.r is x
    else:
        _close("r", got.r, r, tr)
    _close("u", got.u, u, tu)
    _close("post_rstd", got.post_rstd, sy, ty)
    _close("pre_rstd", got.pre_rstd, sr, ts)


def _check_bwd(fwd, y, dr, du, gt, wq, wp, beta, got):
    rows = fwd.r.shape[0]
    ref = R.norm_bwd(fwd, y, dr, du, gt, wq, wp, beta)
    dt = fwd.r.dtype
    for name, g in (("dx", got.dx), ("dy", got.dy)):
        if name in ref:
            v, m = ref[name]
            _close(name, g, v, R.BWD * m + R.half(dt) * (v.abs() + R.BWD * m))
        else:
            assert g is None
    for name, g in (("d_gate", got.d_gate), ("d_post", got.d_post_weight), ("d_pre", got.d_pre_weight)):
        v, m = ref.get(name, (None, None))
        _close(name, g, v, None if v is None else R.bwd_col_tol(rows) * m + R.E * v.abs())


def _both(T, d, dt, gate, post, pre, beta, with_y=True, with_dr=True, seed=0):
    x, y, gt, wq, wp, dr, du = _inputs(T, d, dt, gate, post, pre, seed, with_y)
    fwd = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp, beta=beta, eps=EPS)
    _check_fwd(x, y, gt, wq, wp, beta, fwd)
    dr = dr if with_dr else None
    got = block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp, beta=beta)
    _check_bwd(fwd, y, dr, du, gt, wq, wp, beta, got)


@pytest.mark.parametrize("gate,post,pre", list(itertools.product(["none", "channel", "token"], [False, True],
                                                                 [False, True])))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(5, 64), (130, 333), (1300, 1280)])
def test_every_form(T, d, dt, gate, post, pre):
    _both(T, d, DT[dt], gate, post, pre, beta=1.25)


# each width of the row kernel (vectors of 16 bytes, single elements), and its borders
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 256, 512, 513, 520, 1000, 1023, 1024, 1025, 2048, 2056, 4095, 4096,
                               4104, 8191, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_every_width(d, dt):
    _both(3, d, DT[dt], "channel", True, True, beta=0.5)


@pytest.mark.parametrize("T", [1, 2, 591, 592, 593, 2000])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_every_length(T, gate):
    _both(T, 72, torch.bfloat16, gate, True, True, beta=1.0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [640, 65])
def test_only_the_norm_before(dt, d):
    _both(77, d, DT[dt], "none", False, True, beta=1.0, with_y=False)
    _both(77, d, DT[dt], "none", False, True, beta=1.0, with_y=False, with_dr=False)


# rows that start anywhere within 16 bytes, enough of them that each CTA takes several
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(20001, 66), (9000, 131), (7000, 257), (5000, 333), (4000, 511), (3001, 2050),
                                 (3000, 2044), (2500, 2600), (2000, 4091), (1700, 4808), (1500, 5003), (1201, 8170)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_many_rows_that_start_anywhere(T, d, dt, gate):
    _both(T, d, DT[dt], gate, True, True, beta=0.75)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [77, 257, 601, 2101, 4090, 4501])
def test_rows_that_start_anywhere_keep_to_themselves(d, dt):
    x, y, gt, wq, wp, dr, du = _inputs(900, d, DT[dt], "channel", True, True, seed=3)
    want = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp)
    grads = block_norm_backward(want, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp)
    # a row of NaN reaches no other row, in place either
    for row in (0, 451, 899):
        x2, y2 = x.clone(), y.clone()
        x2[row] = float("nan")
        got = block_norm(x2, y2, gate=gt, post_weight=wq, pre_weight=wp,
                         out=BlockNorm(x2, y2, torch.empty_like(want.post_rstd), torch.empty_like(want.pre_rstd)))
        others = torch.arange(900, device="cuda") != row
        for a, b in zip(got, want):
            assert torch.equal(a[others], b[others])
        assert bool(got.r[row].isnan().all()) and bool(got.u[row].isnan().all())
        du2 = du.clone()
        du2[row] = float("nan")
        g2 = block_norm_backward(want, y, dr=dr, du=du2, gate=gt, post_weight=wq, pre_weight=wp)
        assert torch.equal(g2.dx[others], grads.dx[others]) and torch.equal(g2.dy[others], grads.dy[others])
    # parameters and results at any element, and what lies around the rows
    for off in (1, 2, 3):
        p = [torch.empty(d + off, device="cuda")[off:].copy_(t) for t in (gt, wq, wp)]
        got = block_norm(x, y, gate=p[0], post_weight=p[1], pre_weight=p[2])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        g2 = block_norm_backward(want, y, dr=dr, du=du, gate=p[0], post_weight=p[1], pre_weight=p[2])
        assert all(torch.equal(a, b) for a, b in zip(g2, grads))
    room = torch.full((902 * d + 16,), 7.0, dtype=DT[dt], device="cuda")
    at = (d + 7) // 8 * 8   # 16-byte aligned, rows before and behind
    r = room[at:at + 900 * d].view(900, d)
    got = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp,
                     out=BlockNorm(r, torch.empty_like(x), want.post_rstd.clone(), want.pre_rstd.clone()))
    assert torch.equal(got.r, want.r)
    assert bool((room[:at] == 7).all()) and bool((room[at + 900 * d:] == 7).all())


def test_no_gradient_of_the_stream():
    _both(300, 256, torch.bfloat16, "token", True, True, beta=2.0, with_dr=False)


def test_no_rows():
    x, y, gt, wq, wp, dr, du = _inputs(0, 64, torch.bfloat16, "channel", True, True)
    fwd = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp)
    g = block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp)
    assert fwd.r.shape == (0, 64) and g.dx.shape == (0, 64)
    assert not g.d_gate.any() and not g.d_post_weight.any() and not g.d_pre_weight.any()
    x, y, gt, wq, wp, dr, du = _inputs(0, 64, torch.bfloat16, "token", True, True)
    fwd = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp)
    assert block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp).d_gate.shape == (0, 1)


def test_in_place_and_unaligned():
    x, y, gt, wq, wp, dr, du = _inputs(37, 264, torch.bfloat16, "channel", True, True)
    want = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp, eps=EPS)
    xc, yc = x.clone(), y.clone()
    got = block_norm(xc, yc, gate=gt, post_weight=wq, pre_weight=wp, eps=EPS,
                     out=BlockNorm(xc, yc, torch.empty(37, device="cuda"), torch.empty(37, device="cuda")))
    assert got.r is xc and got.u is yc
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # a buffer that starts between two 16-byte boundaries: single elements, other order of sums
    sx = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
    _check_fwd(sx, y, gt, wq, wp, 1.0, block_norm(sx, y, gate=gt, post_weight=wq, pre_weight=wp, eps=EPS))
    sw = torch.empty(265, device="cuda")[1:].copy_(wq)
    _check_fwd(x, y, gt, sw, wp, 1.0, block_norm(x, y, gate=gt, post_weight=sw, pre_weight=wp, eps=EPS))


def test_rows_of_zeros_and_of_one_infinity():
    x, y, gt, wq, wp, dr, du = _inputs(4, 128, torch.float32, "none", True, True)
    x[1], y[1] = 0, 0
    y[2, 5] = float("inf")
    clean = block_norm(x[:2].contiguous(), y[:2].contiguous(), post_weight=wq, pre_weight=wp, eps=EPS)
    got = block_norm(x, y, post_weight=wq, pre_weight=wp, eps=EPS)
    assert torch.equal(got.r[:2], clean.r) and torch.equal(got.u[:2], clean.u)
    assert not got.r[1].any() and not got.u[1].any() and bool(got.r[3].isfinite().all())


def test_gradients_agree_with_differences():
    """fp32, central differences of a scalar of r and u: second-order error h^2 and the forward's
    rounding over h, both far below the bound of 1e-2 of the gradient's scale."""
    T, d, beta, h = 3, 24, 1.5, 2.0 ** -6
    for gate, post, pre in (("channel", True, True), ("token", True, True), ("none", False, True),
                            ("channel", False, False)):
        x, y, gt, wq, wp, dr, du = _inputs(T, d, torch.float32, gate, post, pre, seed=4)

        def loss(x, y, gt, wq, wp):
            o = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp, beta=beta, eps=EPS)
            s = (o.r.double() * dr.double()).sum()
            return float(s + (o.u.double() * du.double()).sum()) if pre else float(s)

        args = [x, y, gt, wq, wp]
        fwd = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp, beta=beta, eps=EPS)
        got = block_norm_backward(fwd, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp, beta=beta)
        for i, g in enumerate(got):
            if args[i] is None:
                assert g is None
                continue
            scale = float(g.abs().max())
            for flat in range(0, args[i].numel(), 7):
                p, m = [t.clone() if t is not None else None for t in args], [
                    t.clone() if t is not None else None for t in args]
                p[i].view(-1)[flat] += h
                m[i].view(-1)[flat] -= h
                num = (loss(*p) - loss(*m)) / (p[i].view(-1)[flat] - m[i].view(-1)[flat]).double().item()
                assert abs(num - float(g.view(-1)[flat])) <= 1e-2 * scale, (gate, i, flat)


def test_repeats_streams_and_graphs_agree_bit_for_bit():
    x, y, gt, wq, wp, dr, du = _inputs(700, 640, torch.bfloat16, "channel", True, True)

    def step(stream=None):
        f = block_norm(x, y, gate=gt, post_weight=wq, pre_weight=wp, stream=stream)
        return (*f, *block_norm_backward(f, y, dr=dr, du=du, gate=gt, post_weight=wq, pre_weight=wp, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for got in (step(), step(side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):   # two graphs, replayed side by side: each call has a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    for _ in range(3):
        for (g, _), s in zip(graphs, (torch.cuda.current_stream(), side)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bindings_refuse():
    x, y, gt, wq, wp, dr, du = _inputs(8, 64, torch.bfloat16, "channel", True, True)
    with pytest.raises(ValueError, match="y must"):
        block_norm(x, y[:4], pre_weight=wp)
    with pytest.raises(ValueError, match="gate"):
        block_norm(x, y, gate=gt.to(torch.bfloat16))
    with pytest.raises(ValueError, match="gate"):
        block_norm(x, y, gate=torch.zeros(8, device="cuda"))     # per token is [T, 1]
    with pytest.raises(ValueError, match="post_weight"):
        block_norm(x, y, post_weight=wq[:32])
    with pytest.raises(RuntimeError, match="neither"):
        block_norm(x)
    with pytest.raises(RuntimeError, match="without y"):
        block_norm(x, pre_weight=wp, beta=2.0)
    with pytest.raises(RuntimeError, match="eps"):
        block_norm(x, y, pre_weight=wp, eps=0.0)
    with pytest.raises(RuntimeError, match="overlap"):
        block_norm(x, y, pre_weight=wp, out=BlockNorm(x, x, None, torch.empty(8, device="cuda")))
    fwd = block_norm(x, y, pre_weight=wp)
    with pytest.raises(ValueError, match="du goes"):
        block_norm_backward(fwd, y, dr=dr, pre_weight=wp)
    with pytest.raises(ValueError, match="dr is required"):
        block_norm_backward(fwd, y)
    with pytest.raises(ValueError, match="post_rstd"):
        block_norm_backward(fwd, y, dr=dr, du=du, post_weight=wq, pre_weight=wp)
