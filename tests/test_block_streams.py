"""What a MoEBlock's layer reads is recorded on the stream it runs on (CPU only: the norms and the
layer are stand-ins, the stream one that notes what it was given)."""
import pytest
import torch

from mixture_experts_layer_65_b200 import block
from mixture_experts_layer_65_b200.block import BlockNorm, BlockNormGrads, MoEBlock, MoEOutput

T, D = 4, 8


class Noted:
    """on_stream's stand-in: the inputs of the calls that are open."""
    open = []

    def __init__(self, device, stream=None, inputs=()):
        self.inputs = list(inputs)

    def __enter__(self):
        Noted.open.append(self)
        return 0

    def __exit__(self, *a):
        Noted.open.remove(self)
        return False


def _recorded(*read):
    given = {t.data_ptr() for on in Noted.open for t in on.inputs if t is not None}
    return all(t.data_ptr() in given for t in read)


class Layer:
    has_bias = True

    def forward_branch(self, u, out=None, stream=None):
        assert _recorded(u)
        return MoEOutput(*(torch.zeros(2) for _ in range(5)))

    def backward_branch(self, u, out, dy, d_aux, weights, stream=None):
        assert _recorded(u, out.topk_idx, out.topk_w, out.expert_counts)
        return tuple(torch.zeros(T, D) for _ in range(6))


def test_the_layers_inputs_are_recorded(monkeypatch):
    def norm(x, y=None, **kw):
        return BlockNorm(x if y is None else torch.zeros(T, D), torch.zeros(T, D), None, torch.zeros(T))

    def norm_backward(*a, **kw):
        return BlockNormGrads(*(torch.zeros(T, D) for _ in range(5)))

    monkeypatch.setattr(block, "block_norm", norm)
    monkeypatch.setattr(block, "block_norm_backward", norm_backward)
    monkeypatch.setattr(block, "on_stream", Noted)
    blk = MoEBlock(Layer(), torch.ones(D))
    x = torch.zeros(T, D)
    out = blk(x)
    blk.backward(out, x)
    given = blk(x, norm_in=norm(x))
    blk.backward(given, x, norm_in_given=True)
    assert not Noted.open


def test_a_norm_of_another_tensor_is_refused(monkeypatch):
    monkeypatch.setattr(block, "block_norm", lambda *a, **kw: pytest.fail("ran"))
    monkeypatch.setattr(block, "on_stream", Noted)
    blk = MoEBlock(Layer(), torch.ones(D))
    x, other = torch.zeros(T, D), torch.zeros(T, D)
    for r in (other, x[1:], x[:3]):
        with pytest.raises(ValueError, match="must be x"):
            blk(x, norm_in=BlockNorm(r, torch.zeros(T, D), None, torch.zeros(T)))
