"""Weight gradients of many tiles while a stream of higher priority keeps the GPU busy with small
kernels: every tile is written, bit for bit as by the call alone (requests for unstarted clusters
may be refused meanwhile)."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build, grouped

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("groups,rows,n,k", [(64, 20, 512, 768), (48, 700, 520, 512), (3, 3000, 1408, 2048)])
def test_every_tile_is_written(groups, rows, n, k):
    g = torch.Generator(device="cuda").manual_seed(1)
    counts = torch.full((groups,), rows, dtype=torch.int32, device="cuda")
    dy = torch.randn(groups * rows, n, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(groups * rows, k, generator=g, device="cuda").to(torch.bfloat16)
    want = grouped.grouped_mm_wgrad(dy, x, counts)
    low, high = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-5)
    small = torch.zeros(1 << 20, device="cuda")
    outs = [torch.empty_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(8):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for o in outs:
            grouped.grouped_mm_wgrad(dy, x, counts, out=o, stream=low)
            with torch.cuda.stream(high):
                for _ in range(30):
                    small.add_(1.0)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)
    grouped.device_status()
