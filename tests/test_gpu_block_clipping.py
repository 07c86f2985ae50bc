"""A MoEBlock's clipping: the norm of its parameters' gradients in 64 bits, rounded once to fp32;
gradients that are no parameter's come back as they are without clipping."""
import pytest
import torch

from mixture_experts_layer_65_b200 import build
from mixture_experts_layer_65_b200 import workloads as W
from mixture_experts_layer_65_b200.block import MoEBlock
from mixture_experts_layer_65_b200.layer import MoELayer
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
SMALL = dict(T=300, d=256, n_shared=2, n_routed=16, inter=192, top_k=4)


@pytest.fixture(scope="module", autouse=True)
def _lib_ready():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("zipf", [None, 0.5], ids=["no_bias", "bias"])
@pytest.mark.parametrize("kind", ["own", "channel", "token"])
def test_the_norm_is_the_parameters(kind, zipf):
    w = W.make_workload("16b_prefill", zipf_s=zipf, **SMALL)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*s, std=1.0, mean=0.0):
        return mean + std * torch.randn(*s, generator=gen, device="cuda")

    layer = MoELayer.from_workload(w)
    layer.backward_prepare()
    d, T = w.d, w.T
    own = rnd(d, std=0.2, mean=0.5)
    given = {"own": None, "channel": rnd(d, std=0.2, mean=0.5), "token": rnd(T, 1, std=0.2, mean=0.5)}[kind]
    blk = MoEBlock(layer, pre_weight=rnd(d, std=0.1, mean=1.0), post_weight=rnd(d, std=0.1, mean=1.0), gate=own)
    x = rnd(T, d, std=2.0).to(torch.bfloat16)
    dr = rnd(T, d).to(torch.bfloat16)

    def step(max_norm):
        out = blk(x, gate=given)
        return blk.backward(out, dr, d_aux=1.0, gate=given, max_norm=max_norm)

    raw = step(None)
    true = [raw.d_post_weight, raw.d_pre_weight, raw.d_centroids, raw.d_w_gate, raw.d_w_up, raw.d_w_down]
    true += [raw.d_gate] if kind == "own" else []
    true += [raw.d_bias] if zipf else []
    norm = R.norm_sq(true) ** 0.5
    got = step(0.25 * norm)
    assert abs(float(got.grad_norm) - norm) <= 1.001 * R.E * norm
    kept = ["dx"] + (["d_gate"] if kind != "own" else []) + (["d_bias"] if not zipf else [])
    scaled = ["d_post_weight", "d_pre_weight", "d_centroids", "d_w_gate", "d_w_up", "d_w_down"]
    scaled += [n for n in ("d_gate", "d_bias") if n not in kept]
    for n in kept:
        assert torch.equal(getattr(got, n), getattr(raw, n)), n
    for n in scaled:   # at most the coefficient, the product and max_norm rounded to fp32
        ref = getattr(raw, n).double() * 0.25
        assert bool(((getattr(got, n).double() - ref).abs() <= 3.01 * R.E * ref.abs() + 1e-44).all()), n
    layer.device_status()
