"""The gradient norm and clipping on the GPU against 64-bit sums.

The norm: 64-bit squares and sums, rounded once to fp32 (half a step, 2^-24; the 64-bit sums'
own error is below 1e-12).  A clipped value: the coefficient rounded to fp32, the product
rounded to fp32 and, for bf16, once more: 2 * 2^-24 + half a step of the type; values below
the type's smallest normal number are off by at most half of its smallest step."""
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


def _grads(sizes, dts, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(*s, generator=g, device="cuda") * std).to(dt) for s, dt in zip(sizes, dts)]


def _check(grads, before, norm, max_norm):
    want = math.sqrt(R.norm_sq(before))
    assert norm.shape == (1,) and norm.dtype == F32
    assert abs(float(norm) - want) <= 1.001 * R.E * want
    c = max_norm / want if want > max_norm else 1.0
    for g, b in zip(grads, before):
        if c == 1.0:
            assert torch.equal(g, b)
            continue
        ref = b.double() * c
        tiny = torch.finfo(g.dtype).smallest_normal * torch.finfo(g.dtype).eps
        tol = (2.001 * R.E + (R.half(BF) if g.dtype == BF else 0)) * ref.abs() + tiny
        assert bool(((g.double() - ref).abs() <= tol).all())


LISTS = {
    "one": ([(1,)], [F32]),
    "layer": ([(6, 40, 24), (6, 40, 24), (6, 24, 40), (5, 24), (5,)], [F32] * 5),
    "mixed": ([(1,), (0,), (7,), (4096, 9), (3, 3, 3), (1000003,), (0, 5), (32768,), (32769,)],
              [BF, F32, F32, BF, F32, BF, BF, F32, F32]),
    "two_tables": ([(1 + i % 37,) for i in range(2300)], [BF if i % 3 else F32 for i in range(2300)]),
    "at_small_table": ([(5,)] * 48, [F32] * 48),
    "past_small_table": ([(5,)] * 49, [BF] * 49),
    "all_empty": ([(0,), (0, 3)], [F32, BF]),
}


@pytest.mark.parametrize("factor", [0.3, 4.0])
@pytest.mark.parametrize("sizes,dts", LISTS.values(), ids=LISTS.keys())
def test_in_place_and_into_others(sizes, dts, factor):
    before = _grads(sizes, dts)
    max_norm = factor * max(math.sqrt(R.norm_sq(before)), 1e-3)
    grads = [b.clone() for b in before]
    norm = clip.clip_grad_norm(grads, max_norm)
    _check(grads, before, norm, max_norm)
    outs = [torch.full_like(b, float("nan")) for b in before]
    src = [b.clone() for b in before]
    norm2 = clip.clip_grad_norm(src, max_norm, out=outs)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(src, before))
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    assert torch.equal(clip.grad_norm(before), norm)
    # the two steps apart
    s = clip.grad_sumsq(before)
    assert s.dtype == torch.float64 and float(s) == pytest.approx(R.norm_sq(before), rel=1e-12)
    grads = [b.clone() for b in before]
    assert torch.equal(clip.scale_grads(grads, s, max_norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))


def test_views_of_one_buffer_at_every_offset():
    for dt in (BF, F32):
        flat = _grads([(9000,)], [dt])[0]
        cuts = [0, 1, 3, 10, 25, 26, 61, 400, 777, 2001, 2002, 8999, 9000]
        want = flat.clone()
        parts = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        norm = clip.clip_grad_norm(parts, 1.0)
        _check([flat], [want], norm, 1.0)
        # into a buffer with another offset from a 16-byte boundary: single elements
        other = torch.empty(9001, dtype=dt, device="cuda")[1:]
        flat.copy_(want)
        clip.clip_grad_norm(parts, 1.0, out=[other[a:b] for a, b in zip(cuts, cuts[1:])])
        _check([other], [want], norm, 1.0)


def test_neighbours_keep_their_values():
    buf = torch.full((1 << 16,), 5.0, device="cuda")
    g = buf[1001:40007]
    g.normal_()
    clip.clip_grad_norm([g], 0.01)
    assert bool((buf[:1001] == 5).all()) and bool((buf[40007:] == 5).all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("scale", [1e-30, 1e25])
def test_squares_outside_the_fp32_range(dt, scale):
    before = _grads([(1000,), (33,)], [dt, dt], std=scale)
    grads = [b.clone() for b in before]
    norm = clip.clip_grad_norm(grads, 0.5 * scale)
    _check(grads, before, norm, float(torch.tensor(0.5 * scale)))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(value):
    before = _grads([(100,), (50,)], [F32, BF])
    before[1][7] = value
    grads = [b.clone() for b in before]
    norm = clip.clip_grad_norm(grads, 1.0)
    assert not math.isfinite(float(norm))
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(grads, before))
    outs = [torch.zeros_like(b) for b in before]
    clip.clip_grad_norm(grads, 1.0, out=outs)
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(outs, before))


def test_limits_of_zero_and_infinity():
    before = _grads([(100,)], [F32])
    g = [before[0].clone()]
    clip.clip_grad_norm(g, float("inf"))
    assert torch.equal(g[0], before[0])
    clip.clip_grad_norm(g, 0.0)
    assert not g[0].any()
    assert float(clip.clip_grad_norm(g, 0.0)) == 0.0       # a norm of zero is within any limit


def test_repeats_streams_and_graphs_agree_bit_for_bit():
    before = _grads([(300, 70), (11,), (100001,)], [F32, BF, BF])
    outs = [torch.empty_like(b) for b in before]
    want = clip.clip_grad_norm(before, 2.0, out=outs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs2 = [torch.empty_like(b) for b in before]
    torch.cuda.synchronize()
    norm = clip.clip_grad_norm(before, 2.0, out=outs2, stream=side)
    side.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, outs2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip.clip_grad_norm(before, 2.0, out=outs2)
    for _ in range(2):
        for o in outs2:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, outs2))


def test_bindings_refuse():
    g = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        clip.clip_grad_norm([g.t()[1:]], 1.0)
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        clip.clip_grad_norm([g, g.double()], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        clip.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError, match="elements"):
        clip.clip_grad_norm([g], 1.0, out=[torch.zeros(63, device="cuda")])
    with pytest.raises(ValueError, match="type"):
        clip.clip_grad_norm([g], 1.0, out=[torch.zeros(64, dtype=BF, device="cuda")])
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        clip.clip_grad_norm([g, None], 1.0)
    with pytest.raises(ValueError, match=r"out\[0\]"):
        clip.clip_grad_norm([g], 1.0, out=[g.cpu()])
    with pytest.raises(RuntimeError, match="shares memory"):
        clip.clip_grad_norm([g, g], 1.0)
    with pytest.raises(RuntimeError, match="max_norm"):
        clip.clip_grad_norm([g], -1.0)
    with pytest.raises(ValueError, match="sumsq"):
        clip.scale_grads([g], torch.zeros(1, device="cuda"), 1.0)
