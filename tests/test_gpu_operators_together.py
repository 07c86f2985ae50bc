"""The training-side operators as they are used together: a MoEBlock (norm, layer, gate and
residual, next norm) forward and backward with clipping, and experts of one's own between the
expert-parallel dispatch and combine.

Tolerances: each norm by its own (tests/operators_ref.py) from the tensors it was given; the
layer's output and gradients like the layer's own tests, max|x - x_ref| <= 2e-2 max|x_ref|
(at most four bf16 roundings on a path)."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_65_b200 import build, grouped
from mixture_experts_layer_65_b200 import workloads as W
from mixture_experts_layer_65_b200.block import MoEBlock, block_norm
from mixture_experts_layer_65_b200.expert_parallel import LibEPBackend
from mixture_experts_layer_65_b200.layer import MoELayer, to_device_tensor
from oracle import moe_oracle as O
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
SMALL = dict(d=256, n_shared=2, n_routed=16, inter=192, top_k=4)
TOL = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _near(got, ref, tol=TOL):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    err = float(np.abs(got - ref).max()) / max(float(np.abs(ref).max()), 1e-30)
    assert err <= tol, err


def _close(got, ref, tol):
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("T", [300, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_forward_branch_is_the_forward_without_its_input(T, e4m3):
    w = W.make_workload("16b_prefill", T=T, gate_up_e4m3=e4m3, **SMALL)
    layer = MoELayer.from_workload(w)
    u = to_device_tensor(w.u, "cuda")
    full, part = layer.forward(u), layer.forward_branch(u)
    layer.device_status()
    assert torch.equal(full.topk_idx, part.topk_idx) and torch.equal(full.aux_loss, part.aux_loss)
    # h = bf16(u + y), y' = bf16(y): half a step of each
    h, y = full.h.double(), part.h.double()
    tol = R.half(torch.bfloat16) * (h.abs() + y.abs()) * 1.01 + 1e-6
    assert bool(((h - (u.double() + y)).abs() <= tol).all())


def test_forward_branch_of_an_fp32_layer():
    w = W.make_workload("tiny")
    layer = MoELayer.from_workload(w)
    u = to_device_tensor(w.u, "cuda")
    full, part = layer.forward(u).h.double(), layer.forward_branch(u).h.double()
    assert bool(((full - (u.double() + part)).abs() <= 8 * R.E * (full.abs() + part.abs() + u.double().abs())).all())


def _block(T=300, seed=5, next_weight=True):
    w = W.make_workload("16b_prefill", T=T, **SMALL)
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = w.d

    def rnd(*s, std=1.0, mean=0.0):
        return mean + std * torch.randn(*s, generator=g, device="cuda")

    layer = MoELayer.from_workload(w)
    blk = MoEBlock(layer, pre_weight=rnd(d, std=0.1, mean=1.0), post_weight=rnd(d, std=0.1, mean=1.0),
                   gate=rnd(d, std=0.2, mean=0.5), beta=1.25)
    nw = rnd(d, std=0.1, mean=1.0) if next_weight else None
    x = rnd(T, d, std=2.0).to(torch.bfloat16)
    dr, du = rnd(T, d).to(torch.bfloat16), rnd(T, d).to(torch.bfloat16)
    return w, blk, nw, x, dr, du


def _oracle_grads(w, u, dy, d_aux):
    g = O.moe_backward(_bits(u), w.centroids, w.w_gate, w.w_up, w.w_down, w.n_shared, w.top_k, w.alpha1,
                       dy.double().cpu().numpy(), d_aux=d_aux)
    return g, g.du - dy.double().cpu().numpy()      # without the layer's own residual


def test_block_forward_and_backward():
    w, blk, nw, x, dr, du = _block()
    blk.layer.backward_prepare()
    out = blk(x, next_weight=nw)
    # the norm before, from x
    _, u, _, sr, _ = R.norm_fwd(x, None, None, None, blk.pre_weight, 1.0, blk.eps)
    _, tu, _, ts = R.norm_fwd_tol(x, None, None, None, blk.pre_weight, 1.0, blk.eps, x.dtype)
    _close(out.norm_in.u, u, tu)
    _close(out.norm_in.pre_rstd, sr, ts)
    # the layer on that input
    ref = O.moe_forward(_bits(out.norm_in.u), w.centroids, w.w_gate, w.w_up, w.w_down, w.n_shared, w.top_k, w.alpha1)
    _near(out.layer.h, ref.h - O.widen(_bits(out.norm_in.u)))
    # the step after, from the layer's output
    args = (x, out.layer.h, blk.gate, blk.post_weight, nw, blk.beta, blk.eps)
    r, un, sy, sr, _ = R.norm_fwd(*args)
    tr, tun, ty, ts = R.norm_fwd_tol(*args, x.dtype)
    for got, v, t in ((out.r, r, tr), (out.norm_out.u, un, tun), (out.norm_out.post_rstd, sy, ty),
                      (out.norm_out.pre_rstd, sr, ts)):
        _close(got, v, t)
    # backward: the same chain the other way
    got = blk.backward(out, dr, du, d_aux=1.0, next_weight=nw)
    blk.layer.device_status()
    after = R.norm_bwd(out.norm_out, out.layer.h, dr, du, blk.gate, blk.post_weight, nw, blk.beta)
    for name, t in (("d_gate", got.d_gate), ("d_post", got.d_post_weight), ("d_pre", got.d_next_weight)):
        v, m = after[name]
        _close(t, v, R.bwd_col_tol(x.shape[0]) * m)
    dy = after["dy"][0].to(torch.bfloat16)
    g, du_layer = _oracle_grads(w, out.norm_in.u, dy, 1.0)
    for t, v in ((got.d_centroids, g.d_centroids), (got.d_bias, g.d_bias), (got.d_w_gate, g.d_w_gate),
                 (got.d_w_up, g.d_w_up), (got.d_w_down, g.d_w_down)):
        _near(t, v)
    before = R.norm_bwd(out.norm_in, None, after["dx"][0].to(torch.bfloat16),
                        torch.from_numpy(du_layer).cuda(), None, None, blk.pre_weight, 1.0)
    _near(got.dx, before["dx"][0].cpu().numpy())
    _near(got.d_pre_weight, before["d_pre"][0].cpu().numpy())
    assert got.du is None and got.grad_norm is None


def test_two_blocks_in_a_row_fused_or_apart():
    """The norm between two blocks in one kernel with the step before it, or on its own."""
    w, a, nw, x, dr, _ = _block()
    _, b, _, _, _, _ = _block(seed=8)
    b.pre_weight = nw
    for blk in (a, b):
        blk.layer.backward_prepare()
    o1 = a(x, next_weight=nw)
    o2 = b(o1.r, norm_in=o1.norm_out)
    p1 = a(x)
    assert torch.equal(p1.r, o1.r)
    p2 = b(p1.r)
    # apart, the norm reads r rounded to bf16: u may differ by a bf16 step of its input's error
    u, v = o1.norm_out.u.double(), p2.norm_in.u.double()
    assert bool(((u - v).abs() <= 4 * R.half(torch.bfloat16) * (u.abs() + 0.1)).all())
    a(x, next_weight=nw)   # the layer's latest forward is the one whose backward runs
    b(o1.r, norm_in=o1.norm_out)
    g2 = b.backward(o2, dr, norm_in_given=True)
    assert g2.du is not None and g2.d_pre_weight is None
    g1 = a.backward(o1, g2.dx, g2.du, next_weight=nw)
    # the same by one norm after the other
    from mixture_experts_layer_65_b200.block import block_norm_backward
    mid = block_norm_backward(o1.norm_out._replace(post_rstd=None), None, dr=g2.dx, du=g2.du, pre_weight=nw)
    apart = block_norm_backward(o1.norm_out._replace(pre_rstd=None), o1.layer.h, dr=mid.dx, gate=a.gate,
                                post_weight=a.post_weight, beta=a.beta)
    _near(g1.d_gate, apart.d_gate.double().cpu().numpy(), 1e-2)
    _near(g1.d_next_weight, mid.d_pre_weight.double().cpu().numpy(), 1e-5)
    with pytest.raises(ValueError, match="no u"):
        b(o1.r, norm_in=p1.norm_out)


def test_a_step_clips_every_parameter_and_can_be_captured():
    w, blk, nw, x, dr, du = _block(T=333)
    blk.layer.backward_prepare()

    def step(stream=None, max_norm=0.5):
        out = blk(x, next_weight=nw, stream=stream)
        return out, blk.backward(out, dr, du, d_aux=1.0, next_weight=nw, max_norm=max_norm, stream=stream)

    _, raw = step(max_norm=None)
    raw = [t.clone() for t in raw.parameters()]
    out, got = step()
    norm = R.norm_sq(raw) ** 0.5
    assert len(raw) == 9 and abs(float(got.grad_norm) - norm) <= 1.001 * R.E * norm
    for t, v in zip(got.parameters(), raw):
        ref = v.double() * (0.5 / norm)
        assert bool(((t.double() - ref).abs() <= 2.01 * R.E * ref.abs() + 1e-44).all())
    want = [t.clone() for t in (out.r, got.dx, got.grad_norm, *got.parameters())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out.r, got.dx, got.grad_norm, *got.parameters()), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out.r, got.dx, got.grad_norm, *got.parameters()), want))
    blk.layer.device_status()


def test_backwards_belong_to_their_forwards():
    w, blk, nw, x, dr, du = _block(T=300)
    layer = blk.layer
    layer.backward_prepare()
    u = block_norm(x, pre_weight=blk.pre_weight).u
    o = layer.forward(u)
    with pytest.raises(RuntimeError, match="moe_forward_branch"):
        layer.backward_branch(u, o, dr)
    o = layer.forward_branch(u)
    with pytest.raises(RuntimeError, match="moe_forward first"):
        layer.backward(u, o, dr)


def test_decode_sized_block():
    w, blk, nw, x, _, _ = _block(T=3)
    out = blk(x, next_weight=nw)
    ref = O.moe_forward(_bits(out.norm_in.u), w.centroids, w.w_gate, w.w_up, w.w_down, w.n_shared, w.top_k, w.alpha1)
    _near(out.layer.h, ref.h - O.widen(_bits(out.norm_in.u)))
    blk.layer.device_status()


def _silu(z):
    return z / (1 + (-z).exp())


@pytest.mark.parametrize("T", [40, 700])
def test_own_experts_between_dispatch_and_combine(T):
    """The library's SwiGLU experts, restated with grouped products, agree with moe_ep_experts;
    their gradients with a 64-bit restatement."""
    w = W.make_workload("16b_prefill", T=T, **SMALL)
    dev = "cuda"
    wg, wu, wd = (to_device_tensor(t, dev) for t in (w.w_gate, w.w_up, w.w_down))
    ep = LibEPBackend(T=w.T, d=w.d, n_routed=w.n_routed, n_shared=w.n_shared, top_k=w.top_k, inter=w.inter,
                      alpha1=w.alpha1, centroids=to_device_tensor(w.centroids, dev), w_gate=wg, w_up=wu, w_down=wd,
                      rank=0, world=1)
    u = to_device_tensor(w.u, dev)
    idx, gates, counts, _, rows = ep.dispatch(u)
    n = rows.shape[0]
    lib_rows = ep.experts(rows, counts.view(1, -1), n)
    ns = w.n_shared
    rg, ru, rd = (t[ns:].contiguous() for t in (wg, wu, wd))
    a, b = grouped.grouped_mm(rows, rg, counts), grouped.grouped_mm(rows, ru, counts)
    hid = (_silu(a.float()) * b.float()).to(torch.bfloat16)
    y = grouped.grouped_mm(hid, rd, counts)
    _near(y, lib_rows.double().cpu().numpy())
    _near(ep.combine(u, y, gates), ep.combine(u, lib_rows, gates).double().cpu().numpy())
    # backward of sum(dy . y) through the three products
    dy = torch.randn(n, w.d, device=dev).to(torch.bfloat16)
    dhid = grouped.grouped_mm_dgrad(dy, rd, counts).float()
    s = torch.sigmoid(a.float())
    da = (dhid * b.float() * s * (1 + a.float() * (1 - s))).to(torch.bfloat16)
    db = (dhid * a.float() * s).to(torch.bfloat16)
    dx = grouped.grouped_mm_dgrad(da, rg, counts).float() + grouped.grouped_mm_dgrad(db, ru, counts).float()
    dwd = grouped.grouped_mm_wgrad(dy, hid, counts)
    dwg = grouped.grouped_mm_wgrad(da, rows, counts)
    grouped.device_status()
    ep.device_status()
    at = 0
    for e, c in enumerate(counts.tolist()):
        x64 = rows[at:at + c].double().requires_grad_()
        g64, u64, d64 = (t[e].double().requires_grad_() for t in (rg, ru, rd))
        (_silu(x64 @ g64.t()) * (x64 @ u64.t()) @ d64.t()).backward(dy[at:at + c].double())
        if c:
            _near(dx[at:at + c], x64.grad.cpu().numpy())
            _near(dwg[e], g64.grad.cpu().numpy())
            _near(dwd[e], d64.grad.cpu().numpy())
        else:
            assert not dwg[e].any() and not dwd[e].any()
        at += c
