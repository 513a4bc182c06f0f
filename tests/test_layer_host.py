"""The attention layer's use of its norm, on the CPU: the operator replaced by a stand-in."""
import copy
import pickle

import pytest
import torch
from torch import nn

from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import LayerNorm, MultiScaleDeformableAttention


@pytest.fixture
def operands(monkeypatch):
    """The sampling operator and the layer norm's launch replaced by CPU arithmetic."""
    def sample(v, shapes, starts, loc, logits, accum, softmax):
        B, Q = loc.shape[:2]
        return v.mean(1).reshape(B, 1, -1).expand(B, Q, -1) + loc.mean(dim=(2, 3, 4, 5)).unsqueeze(-1)

    def norm(x, weight=None, bias=None, residual=None, eps=1e-5, return_sum=False):
        s = x if residual is None else x + residual
        y = nn.functional.layer_norm(s, s.shape[-1:], weight, bias, eps)
        return (y, s) if return_sum else y

    monkeypatch.setattr(binding, "multi_scale_deformable_attention", sample)
    monkeypatch.setattr(binding, "layer_norm", norm)
    torch.manual_seed(0)
    shapes = torch.tensor([[4, 5], [2, 3]])
    return (torch.randn(2, 7, 16), torch.rand(2, 7, 2), torch.randn(2, 26, 16), shapes, torch.tensor([0, 20]))


class Encoder(MultiScaleDeformableAttention):
    """A user's layer, which has a norm of its own under that name."""

    def __init__(self):
        super().__init__(16, 2, 2, 2)
        self.norm = nn.LayerNorm(16)

    def forward(self, query, *args):
        return self.norm(query + super().forward(query, *args))


def test_a_subclass_keeps_its_own_norm(operands):
    layer = Encoder()
    plain = MultiScaleDeformableAttention(16, 2, 2, 2)
    plain.load_state_dict({k: v for k, v in layer.state_dict().items() if not k.startswith("norm")})
    assert torch.equal(layer(*operands), layer.norm(operands[0] + plain(*operands)))
    with pytest.raises(ValueError, match="norm=True"):
        MultiScaleDeformableAttention.forward(layer, *operands, residual=operands[0])


def test_a_layer_made_with_its_norm(operands):
    layer = MultiScaleDeformableAttention(16, 2, 2, 2, norm=True)
    plain = MultiScaleDeformableAttention(16, 2, 2, 2)
    plain.load_state_dict({k: v for k, v in layer.state_dict().items() if not k.startswith("norm")})
    want = layer.norm(plain(*operands), residual=operands[0])
    assert torch.equal(layer(*operands), want)
    for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        assert torch.equal(other(*operands), want)
    layer.norm = nn.Sequential()         # replaced: called all the same
    with pytest.raises(TypeError):
        layer(*operands)


@pytest.mark.parametrize("norm", [False, True])
def test_layers_pickled_before(operands, norm):
    """States without the mark of how the layer was made: one of before it could have a
    norm, and one with the framework's norm."""
    layer = MultiScaleDeformableAttention(16, 2, 2, 2, norm=norm)
    want = layer(*operands)
    layer.__dict__.pop("ends_in_norm", None)
    if not norm:
        layer.__dict__.pop("norm", None)
        layer._modules.pop("norm", None)
    assert torch.equal(layer(*operands), want)
    assert norm == isinstance(getattr(layer, "norm", None), LayerNorm)
