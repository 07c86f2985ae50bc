"""Which gradients of a MoEBlock are its parameters', and so are clipped (CPU only: the norms, the
layer and the clipping are stand-ins that hand out made-up gradients)."""
import pytest
import torch

from mixture_experts_layer_65_b200 import block
from mixture_experts_layer_65_b200.block import BlockNorm, BlockNormGrads, MoEBlock, MoEBlockGrads, MoEBlockOutput

T, D = 5, 8


class Layer:
    def __init__(self, has_bias):
        self.has_bias = has_bias

    def backward_branch(self, u, out, dy, d_aux, weights, stream=None):
        w = [torch.randn(3, 4) for _ in range(3)] if weights else [None] * 3
        return (torch.randn(T, D), torch.randn(2, D), torch.randn(2), *w)


class NoStream:
    def __init__(self, *a):
        pass

    def __enter__(self):
        return 0

    def __exit__(self, *a):
        return False


@pytest.fixture
def clipped(monkeypatch):
    """What reached the clipping."""
    seen = []

    def norm_backward(fwd, y, *, gate=None, post_weight=None, pre_weight=None, **kw):
        def like(t):
            return None if t is None else torch.randn_like(t)
        return BlockNormGrads(torch.randn(T, D), torch.randn(T, D), like(gate), like(post_weight), like(pre_weight))

    def clip(grads, max_norm, stream=None):
        seen.extend(grads)
        return torch.ones(1)

    monkeypatch.setattr(block, "block_norm_backward", norm_backward)
    monkeypatch.setattr(block, "clip_grad_norm", clip)
    monkeypatch.setattr(block, "on_stream", NoStream)
    return seen


def _backward(has_bias, gate, call_gate, **kw):
    norm = BlockNorm(torch.zeros(T, D), torch.zeros(T, D), None, None)
    layer_out = block.MoEOutput(*(torch.zeros(1) for _ in range(5)))
    blk = MoEBlock(Layer(has_bias), torch.ones(D), torch.ones(D), gate)
    call_gate = gate if call_gate == "own" else call_gate
    return blk.backward(MoEBlockOutput(norm.r, norm, layer_out, norm), torch.zeros(T, D), gate=call_gate,
                        next_weight=torch.ones(D), max_norm=1.0, **kw)


GATES = {   # the block's gate, the call's, whether its gradient is a parameter's
    "none": (None, None, False),
    "own": (torch.ones(D), None, True),
    "own_given_again": (torch.ones(D), "own", True),
    "channel_to_the_call": (torch.ones(D), torch.ones(D), False),
    "token_to_the_call": (None, torch.ones(T, 1), False),
    "token_in_place_of_own": (torch.ones(D), torch.ones(T, 1), False),
    "token_held": (torch.ones(T, 1), None, False),
}


@pytest.mark.parametrize("has_bias", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("gate,call_gate,counts", GATES.values(), ids=GATES.keys())
def test_only_parameters_are_clipped(clipped, has_bias, weights, gate, call_gate, counts):
    g = _backward(has_bias, gate, call_gate, weights=weights)
    want = [g.d_gate if counts else None, g.d_post_weight, g.d_pre_weight, g.d_next_weight, g.d_centroids,
            g.d_bias if has_bias else None, g.d_w_gate, g.d_w_up, g.d_w_down]
    want = {t.data_ptr() for t in want if t is not None}
    assert {t.data_ptr() for t in clipped if t.numel()} == want
    assert {t.data_ptr() for t in g.parameters() if t.numel()} == want
    # the places are those of the gradients that there are
    assert len(g.parameters()) == sum(t is not None for t in g[2:11])
    assert g.d_bias.numel() > 0 and (g.d_gate is None) == (gate is None and call_gate is None)


def test_gradients_made_by_hand_are_all_parameters():
    g = MoEBlockGrads(*(torch.ones(2) for _ in range(12)))
    assert len(g.parameters()) == 9 and all(t.numel() == 2 for t in g.parameters())
