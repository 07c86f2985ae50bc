"""Refusals of the handle-less operators (grouped products, block norms, gradient clipping):
bad arguments are turned away before a GPU is touched (CPU only)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_65_b200 import _lib, block, build, clip, grouped

BAD, UNSUP = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
A = 1 << 20   # made-up addresses far apart: refused calls never read them
B, C, D = 2 << 40, 3 << 40, 4 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


GROUPED = dict(a=A, b=B, counts=C, g=4, rows=64, n=64, k=64, dtype=_lib.MOE_BF16, out=D)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), BAD), (dict(b=None), BAD), (dict(counts=None), BAD), (dict(out=None), BAD),
    (dict(g=0), UNSUP), (dict(g=1025), UNSUP), (dict(rows=-1), BAD), (dict(rows=1 << 30), UNSUP),
    (dict(n=0), BAD), (dict(k=-3), BAD), (dict(n=(1 << 20) + 1), UNSUP), (dict(dtype=2), BAD),
    (dict(dtype=7), BAD), (dict(a=A + 1), BAD), (dict(counts=C + 2), BAD),
    (dict(out=A), BAD), (dict(out=A + 64), BAD), (dict(out=B + 128), BAD), (dict(counts=D + 4), BAD),
    (dict(rows=(1 << 30) - 1, n=1 << 20), UNSUP), (dict(rows=1 << 28), UNSUP), (dict(rows=(1 << 28) - 1, a=None), BAD),
])
@pytest.mark.parametrize("op", ["moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad"])
def test_grouped_products_refuse(L, op, kw, status):
    v = {**GROUPED, **kw}
    args = [v["a"], v["b"], v["counts"], v["g"], v["rows"], v["n"], v["k"], v["dtype"]]
    args += [0, v["out"], None, 0] if op.endswith("wgrad") else [v["out"]]
    assert getattr(L, op)(*args, None) == status
    assert len(L.moe_last_error()) > 0


def test_grouped_products_of_no_rows_do_nothing(L):
    assert L.moe_grouped_mm(None, B, C, 4, 0, 64, 64, _lib.MOE_BF16, None, None) == _lib.MOE_OK
    assert L.moe_grouped_mm_dgrad(None, B, C, 4, 0, 64, 64, _lib.MOE_FP32, None, None) == _lib.MOE_OK


def test_split_weight_gradients_want_their_workspace(L):
    for dt in (_lib.MOE_BF16, _lib.MOE_FP32):
        assert L.moe_grouped_wgrad_workspace(64, 49152, 1408, 2048, dt) == 0       # tiles enough
        assert L.moe_grouped_wgrad_workspace(2, 300, 64, 64, dt) == 0              # rows too few
        size = L.moe_grouped_wgrad_workspace(2, 65536, 64, 64, dt)
        assert size > 2 * 64 * 64 * 4
        args = [A, B, C, 2, 65536, 64, 64, dt, 0, D]
        assert L.moe_grouped_mm_wgrad(*args, None, 0, None) == BAD
        assert L.moe_grouped_mm_wgrad(*args, D + (1 << 30), 2 * 64 * 64 * 4, None) == BAD   # one part's
        assert L.moe_grouped_mm_wgrad(*args, D + (1 << 30) + 4, size, None) == BAD
        assert L.moe_grouped_mm_wgrad(*args, D, size, None) == BAD                 # on the output
        assert L.moe_grouped_mm_wgrad(*args, A + 64, size, None) == BAD            # on an input
    assert L.moe_grouped_wgrad_workspace(0, 65536, 64, 64, 1) == 0                 # refused shapes
    assert L.moe_grouped_wgrad_workspace(2, 0, 64, 64, 1) == 0


E = 5 << 40
NORM = dict(x=A, y=B, gate=None, kind=0, post=C, pre=C, T=8, d=64, dtype=_lib.MOE_BF16, beta=1.0, eps=1e-6,
            r=D, u=D + (1 << 30), ps=E, qs=E + 4096)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(r=None), BAD), (dict(u=None), BAD), (dict(pre=None), BAD),
    (dict(post=None), BAD), (dict(ps=None), BAD), (dict(qs=None), BAD), (dict(y=None), BAD),
    (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(d=0), BAD), (dict(d=16385), UNSUP),
    (dict(dtype=3), BAD), (dict(kind=3), BAD), (dict(kind=1), BAD), (dict(gate=C), BAD),
    (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(beta=float("inf")), BAD), (dict(x=A + 1), BAD), (dict(u=D), BAD), (dict(u=D + 16), BAD),
    (dict(r=A + 128), BAD), (dict(u=B + 2), BAD), (dict(ps=C), BAD), (dict(qs=E + 4), BAD), (dict(qs=D + 64), BAD),
    (dict(r=C - 8), BAD), (dict(u=C + 252), BAD), (dict(gate=D + 8, kind=1), BAD), (dict(gate=D + 4, kind=2), BAD),
    (dict(y=None, r=None, post=None, ps=None, beta=2.0), BAD),
    (dict(y=None, r=None, post=None, ps=None, gate=C, kind=1), BAD),
    (dict(y=None, r=None, post=None, ps=None, pre=None, u=None, qs=None), BAD),
])
def test_block_norm_refuses(L, kw, status):
    v = {**NORM, **kw}
    assert L.moe_block_norm(*[v[n] for n in ("x", "y", "gate", "kind", "post", "pre", "T", "d", "dtype",
                                             "beta", "eps", "r", "u", "ps", "qs")], None) == status
    assert len(L.moe_last_error()) > 0


BWD = dict(y=A, r=B, dr=C, du=C + (1 << 30), gate=None, kind=0, post=C, pre=C, ps=C, qs=C, T=8, d=64,
           dtype=_lib.MOE_FP32, beta=1.0, dx=D, dy=D + (1 << 30), dg=None, dpost=E, dpre=E + 4096, ws=E + 8192,
           size=1 << 20)


@pytest.mark.parametrize("kw", [
    dict(r=None), dict(du=None), dict(dx=None), dict(dy=None), dict(y=None), dict(ps=None), dict(qs=None),
    dict(dpost=None), dict(dpre=None), dict(dg=A), dict(ws=None), dict(size=8 * 64 * 8 - 1), dict(ws=E + 8196),
    dict(pre=None, du=None, qs=None, dpre=None, dr=None), dict(dx=B + 4), dict(dy=D + 8), dict(dy=D),
    dict(kind=1, gate=C), dict(d=0), dict(dtype=9), dict(beta=float("nan")),
    dict(dpost=C), dict(dpre=E), dict(ws=E), dict(ws=D + 16), dict(kind=2, gate=E + (1 << 20), dg=E + (1 << 20)),
    dict(post=D + 16), dict(pre=D + (1 << 30)), dict(ps=D), dict(qs=D + 64), dict(kind=2, gate=D, dg=E + (1 << 20)),
])
def test_block_norm_backward_refuses(L, kw):
    v = {**BWD, **kw}
    got = L.moe_block_norm_backward(*[v[n] for n in (
        "y", "r", "dr", "du", "gate", "kind", "post", "pre", "ps", "qs", "T", "d", "dtype", "beta", "dx", "dy",
        "dg", "dpost", "dpre", "ws", "size")], None)
    assert got == BAD
    assert L.moe_block_norm_workspace(8, 64) == 8 * 64 * 8
    assert L.moe_block_norm_workspace(0, 64) == 0 and L.moe_block_norm_workspace(8, 1 << 20) == 0


def _tables(ptrs, numels, dtypes):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numels), (ctypes.c_int32 * n)(*dtypes))


@pytest.mark.parametrize("ptrs,outs,numels,dtypes", [
    ([A, None], [A, B], [4, 4], [0, 0]),          # NULL gradients
    ([A, B], [A, None], [4, 4], [0, 0]),          # NULL output
    ([A, B], [A, B], [4, -1], [0, 0]),
    ([A, B], [A, B], [4, 4], [0, 2]),             # e4m3 rows are not gradients
    ([A + 2, B], [A + 2, B], [4, 4], [0, 0]),     # fp32 at an odd half-word
    ([A, B], [A + 4, B], [4, 4], [0, 0]),         # shifted against itself
    ([A, A], [A, A], [4, 4], [0, 0]),             # the same buffer twice
    ([A, B], [C, C + 8], [4, 4], [0, 0]),         # outputs overlap
    ([A, B], [B, C], [4, 4], [0, 0]),             # an output is another's gradients
    ([A, A + 8], [A, A + 8], [4, 4], [0, 0]),     # neighbours that overlap
    ([A, A], [A, B], [4, 4], [0, 0]),             # one read while the other is scaled in place
])
def test_clipping_refuses_bad_tables(L, ptrs, outs, numels, dtypes):
    p, n, d = _tables(ptrs, numels, dtypes)
    o = (ctypes.c_void_p * len(outs))(*outs)
    size = L.moe_grad_workspace(len(ptrs))
    assert L.moe_clip_grad_norm(p, o, n, d, len(ptrs), 1.0, D, D + 64, size, None) == BAD
    assert L.moe_grad_scale(p, o, n, d, len(ptrs), D, 1.0, None, None) == BAD


def test_clipping_refuses_results_and_workspaces_on_the_tensors(L):
    p, n, d = _tables([A], [100], [0])
    o = (ctypes.c_void_p * 1)(B)
    size = L.moe_grad_workspace(1)
    for norm, ws in ((A + 8, D), (B + 8, D), (D, A), (D, B - size + 8), (D, B), (D + 8, D)):
        assert L.moe_clip_grad_norm(p, o, n, d, 1, 1.0, norm, ws, size, None) == BAD
    for sumsq, norm, ws in ((A, None, D), (None, A + 4, D), (D, None, A + 392), (D, D + 4, C), (D, None, D)):
        assert L.moe_grad_sumsq(p, n, d, 1, sumsq, norm, ws, size, None) == BAD
    for sumsq, norm in ((B, D), (D, B + 396), (D, A), (D, D + 4)):
        assert L.moe_grad_scale(p, o, n, d, 1, sumsq, 1.0, norm, None) == BAD


def test_clipping_refuses_bad_scalars(L):
    p, n, d = _tables([A], [4], [0])
    size = L.moe_grad_workspace(1)
    for norm in (-1.0, float("nan")):
        assert L.moe_clip_grad_norm(p, p, n, d, 1, norm, D, D + 64, size, None) == BAD
        assert L.moe_grad_scale(p, p, n, d, 1, D, norm, None, None) == BAD
    assert L.moe_clip_grad_norm(p, p, n, d, 1, 1.0, None, D, size, None) == BAD
    assert L.moe_clip_grad_norm(p, p, n, d, 1, 1.0, D, None, size, None) == BAD
    assert L.moe_clip_grad_norm(p, p, n, d, 1, 1.0, D, D + 64, size - 1, None) == BAD
    assert L.moe_clip_grad_norm(p, p, n, d, -1, 1.0, D, D + 64, size, None) == BAD
    assert L.moe_clip_grad_norm(p, None, n, d, 1, 1.0, D, D + 64, size, None) == BAD
    assert L.moe_grad_sumsq(p, n, d, 1, None, None, D, size, None) == BAD
    assert L.moe_grad_sumsq(None, n, d, 1, D, None, D, size, None) == BAD
    assert L.moe_grad_scale(p, p, n, d, 1, None, 1.0, None, None) == BAD


def test_bindings_refuse_host_and_misshapen_tensors():
    x, w = torch.zeros(8, 16), torch.zeros(2, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        grouped.grouped_mm(x, w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        grouped.grouped_mm_wgrad(x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        block.block_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        clip.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        clip.grad_norm([])
