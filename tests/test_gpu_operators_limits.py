"""The training-side operators where a call can go wrong for its surroundings: the first call of
a process inside a graph capture, calls at once on two streams, tensors past 2^31 elements."""
import subprocess
import sys

import pytest
import torch

from mixture_experts_layer_65_b200 import block, build, clip, grouped
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


FIRST = """
import torch
from mixture_experts_layer_65_b200 import block, clip, grouped
d = "cuda"
x = torch.randn(300, 264, device=d).bfloat16()
dy = torch.randn(300, 136, device=d).bfloat16()
w = torch.randn(3, 136, 264, device=d).bfloat16()
c = torch.tensor([100, 0, 190], dtype=torch.int32, device=d)
p = torch.rand(264, device=d)

def run():
    f = block.block_norm(x, x.clone(), gate=p, post_weight=p, pre_weight=p)
    g = block.block_norm_backward(f, x, dr=x, du=x, gate=p, post_weight=p, pre_weight=p)
    outs = [torch.empty(136, 264, device=d), torch.empty(264, device=d)]
    n = clip.clip_grad_norm([w[0].float(), p], 0.5, out=outs)
    y, z = torch.zeros(300, 136, device=d).bfloat16(), torch.zeros(300, 264, device=d).bfloat16()
    return [*f, *g, n, *outs, grouped.grouped_mm(x, w, c, out=y), grouped.grouped_mm_dgrad(dy, w, c, out=z),
            grouped.grouped_mm_wgrad(dy, x, c), grouped.grouped_mm(x.float(), w.float(), c, out=y.float()),
            grouped.grouped_mm_wgrad(dy[:, :33].contiguous(), x[:, :35].contiguous(), c)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
grouped.device_status("cuda")
print("captured")
"""


def test_the_first_call_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_calls_at_once_on_two_streams():
    g = torch.Generator(device="cuda").manual_seed(2)
    counts = torch.tensor([700, 3, 0, 1500, 800, 90], dtype=torch.int32, device="cuda")
    rows = 3093
    sets = []
    for _ in range(2):
        x = torch.randn(rows, 512, generator=g, device="cuda").to(BF)
        dy = torch.randn(rows, 768, generator=g, device="cuda").to(BF)
        w = torch.randn(6, 768, 512, generator=g, device="cuda").to(BF)
        p = torch.rand(512, generator=g, device="cuda")
        sets.append((x, dy, w, p))

    def run(s, stream=None):
        x, dy, w, p = s
        f = block.block_norm(x, x, gate=p, post_weight=p, pre_weight=p, stream=stream)
        b = block.block_norm_backward(f, x, dr=x, du=x, gate=p, post_weight=p, pre_weight=p, stream=stream)
        outs = [torch.empty_like(x), torch.empty_like(w)]
        n = clip.clip_grad_norm([x, w], 1.0, out=outs, stream=stream)
        return [*f, *b, n, *outs, grouped.grouped_mm(x, w, counts, stream=stream),
                grouped.grouped_mm_dgrad(dy, w, counts, stream=stream),
                grouped.grouped_mm_wgrad(dy, x, counts, stream=stream)]

    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[], []]
        for i, (s, st) in enumerate(zip(sets, streams)):
            got[i] = run(s, st)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    grouped.device_status()


def test_rows_past_31_bits_of_elements():
    n, k, tail = 64, 2048, 300
    rows = (1 << 31) // k + 1000          # x has more than 2^31 elements
    x = torch.empty(rows, k, dtype=BF, device="cuda").normal_()
    w = torch.randn(2, n, k, device="cuda").to(BF)
    c = torch.tensor([rows - tail, tail], dtype=torch.int32, device="cuda")
    y = grouped.grouped_mm(x, w, c)
    for lo, hi, e in ((rows - tail - 50, rows - tail, 0), (rows - tail, rows, 1), (0, 50, 0)):
        ref, tol = R.grouped("mm", x[lo:hi], w[e:e + 1], torch.tensor([hi - lo]))
        assert bool(((y[lo:hi].double() - ref).abs() <= tol).all())
    dx = grouped.grouped_mm_dgrad(y, w, c)
    ref, tol = R.grouped("dgrad", y[rows - tail:], w[1:], torch.tensor([tail]))
    assert bool(((dx[rows - tail:].double() - ref).abs() <= tol).all())
    dw = grouped.grouped_mm_wgrad(y, x, c)
    ref, tol = R.grouped("wgrad", y[rows - tail:], x[rows - tail:], torch.tensor([tail]))
    assert bool(((dw[1].double() - ref[0]).abs() <= tol[0]).all())
    grouped.device_status()
    # the same buffers as a residual stream
    p = torch.rand(k, device="cuda")
    f = block.block_norm(x, dx, gate=p, post_weight=p, pre_weight=p)
    b = block.block_norm_backward(f, dx, dr=x, du=x, gate=p, post_weight=p, pre_weight=p)
    s = slice(rows - 100, rows)
    part = block.BlockNorm(*(t[s] for t in f))
    r, u, sy, sr, _ = R.norm_fwd(x[s], dx[s], p, p, p, 1.0, 1e-6)
    tr, tu, ty, ts = R.norm_fwd_tol(x[s], dx[s], p, p, p, 1.0, 1e-6, BF)
    assert bool(((part.r.double() - r).abs() <= tr).all()) and bool(((part.u.double() - u).abs() <= tu).all())
    ref = R.norm_bwd(part, dx[s], x[s], x[s], p, p, p, 1.0)
    for got, name in ((b.dx[s], "dx"), (b.dy[s], "dy")):
        v, m = ref[name]
        assert bool(((got.double() - v).abs() <= R.BWD * m + R.half(BF) * (v.abs() + R.BWD * m)).all())
    del f, b, part, dx
    torch.cuda.empty_cache()
    want = sum(float(t.double().square().sum()) for t in x.split(1 << 16)) ** 0.5
    last = x[-1].clone()
    norm = clip.clip_grad_norm([x], 1.0)
    assert abs(float(norm) - want) <= 1.001 * R.E * want
    assert bool(((x[-1].double() - last.double() / want).abs()
                 <= (2.01 * R.E + R.half(BF)) * (last.double() / want).abs() + 1e-42).all())
