"""A MoEBlock on another stream than its inputs': what the layer reads there may be dropped once the
call has returned, and is not handed out while that stream still reads it."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200 import workloads as W
from mixture_experts_layer_65_b200.block import MoEBlock, block_norm
from mixture_experts_layer_65_b200.layer import MoELayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _take(tensors):
    """Tensors of the same sizes, zero: memory the allocator holds free is handed out first."""
    return [torch.zeros(n, dtype=dt, device="cuda") for n, dt in tensors for _ in range(3)]


def _sizes(ts):
    return [(t.shape, t.dtype) for t in ts]


def test_inputs_of_a_delayed_stream_may_be_dropped():
    w = W.make_workload("16b_prefill", T=300, d=256, n_shared=2, n_routed=16, inter=192, top_k=4)
    layer = MoELayer.from_workload(w)
    layer.backward_prepare()
    gen = torch.Generator(device="cuda").manual_seed(0)
    p = torch.rand(w.d, generator=gen, device="cuda") + 0.5
    blk = MoEBlock(layer, pre_weight=p, post_weight=p)
    x = torch.randn(w.T, w.d, generator=gen, device="cuda").to(torch.bfloat16)
    dr = torch.randn(w.T, w.d, generator=gen, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()

    out = blk(x)
    want = [out.r.clone(), *(t.clone() for t in blk.backward(out, dr) if t is not None and torch.is_tensor(t))]
    _take(_sizes([out.r, out.norm_in.pre_rstd, *out.layer]))   # (a kernel's first launch may wait for the GPU)
    del out
    # forward on the side stream, its norm_in from this one
    norm_in = block_norm(x, pre_weight=p)
    sizes = _sizes([norm_in.u, norm_in.pre_rstd])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    r = blk(x, norm_in=norm_in, stream=side).r
    del norm_in
    taken = _take(sizes)
    torch.cuda.synchronize()
    assert torch.equal(r, want[0])
    # forward here, backward on the side stream
    out = blk(x)
    sizes = _sizes([out.r, out.norm_in.u, out.norm_in.pre_rstd, *out.layer, out.norm_out.post_rstd])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = blk.backward(out, dr, stream=side)
    del out, taken
    taken = _take(sizes)
    torch.cuda.synchronize()
    got = [t for t in got if t is not None and torch.is_tensor(t)]
    assert len(got) == len(want) - 1 and all(torch.equal(a, b) for a, b in zip(got, want[1:]))
    layer.device_status()
