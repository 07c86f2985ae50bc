"""A layer's forward and backward on another stream than their inputs': the inputs may be dropped
once the call has returned, and the results are the caller's on either stream."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200 import workloads as W
from mixture_experts_layer_65_b200.layer import MoELayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("branch", [False, True])
def test_dropped_inputs_keep_their_values_until_they_are_read(branch):
    w = W.make_workload("16b_prefill", T=300, d=256, n_shared=2, n_routed=16, inter=192, top_k=4)
    layer = MoELayer.from_workload(w)
    layer.backward_prepare()
    forward = layer.forward_branch if branch else layer.forward
    backward = layer.backward_branch if branch else layer.backward
    gen = torch.Generator(device="cuda").manual_seed(0)
    keep_u = torch.randn(w.T, w.d, generator=gen, device="cuda").to(torch.bfloat16)
    keep_dh = torch.randn(w.T, w.d, generator=gen, device="cuda").to(torch.bfloat16)
    ref = forward(keep_u)
    want = [*(t.clone() for t in ref), *(t.clone() for t in backward(keep_u, ref, keep_dh))]
    side = torch.cuda.Stream()

    def taken():
        return [torch.zeros_like(keep_u) for _ in range(4)]

    u = keep_u.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    out = forward(u, stream=side)
    del u
    first = taken()
    torch.cuda.synchronize()
    dh = keep_dh.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    grads = backward(keep_u, out, dh, stream=side)
    del dh
    second = taken()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*out, *grads), want))
    layer.device_status()
    del first, second


def test_results_lie_where_no_earlier_work_still_reads():
    """Memory that this stream has freed but still reads is not where another stream's results go."""
    w = W.make_workload("16b_prefill", T=300, d=256, n_shared=2, n_routed=16, inter=192, top_k=4)
    layer = MoELayer.from_workload(w)
    u = torch.randn(w.T, w.d, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    layer.forward(u, stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    a = [torch.full((w.T, w.d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(32)]
    b = [torch.empty_like(t) for t in a]
    b[0].copy_(torch.add(a[0], 1, out=b[1]))   # (a kernel's first launch may wait for the GPU)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for t, o in zip(a, b):
        torch.add(t, 1, out=o)
    del a, t, o                            # read by additions that have not started yet
    outs = [layer.forward(u, stream=side) for _ in range(40)]
    torch.cuda.synchronize()
    assert all(bool((t == 4.0).all()) for t in b)
    # and results that this stream still reads are not the other stream's to reuse
    copies = [torch.empty_like(o.h) for o in outs]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for c, o in zip(copies, outs):
        c.copy_(o.h)
    del outs, o
    with torch.cuda.stream(side):
        again = [torch.zeros(w.T, w.d, dtype=torch.bfloat16, device="cuda") for _ in range(40)]
    torch.cuda.synchronize()
    want = layer.forward(u).h
    assert all(torch.equal(c, want) for c in copies)
    del again
