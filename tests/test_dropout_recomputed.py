"""Dropout in a forward that is run again for its backward (activation checkpointing): the
draw of the first time if the caller gives its counter, else an error and no gradient of
another mask. On the CPU, the launches replaced by stand-ins."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention, MultiScaleDeformableAttention
from test_dropout_copies import operands  # noqa: F401


@pytest.fixture
def layers(operands, monkeypatch):  # noqa: F811
    """The two layers' operators in plain torch."""
    def attend(q, k, v, mask=None, scale=None):
        s = torch.einsum("bqmd,bkmd->bmqk", q, k) * q.shape[-1] ** -0.5
        return torch.einsum("bmqk,bkmd->bqmd", s.softmax(-1), v).flatten(2)

    def sample(v, shapes, starts, loc, logits, accum, softmax):
        B, Q = loc.shape[:2]
        return v.mean(1).reshape(B, 1, -1).expand(B, Q, -1) + loc.mean(dim=(2, 3, 4, 5)).unsqueeze(-1)

    def norm(x, weight=None, bias=None, residual=None, eps=1e-5, return_sum=False):
        return torch.nn.functional.layer_norm(x if residual is None else x + residual, x.shape[-1:], weight, bias, eps)

    monkeypatch.setattr(binding, "attention", attend)
    monkeypatch.setattr(binding, "multi_scale_deformable_attention", sample)
    monkeypatch.setattr(binding, "layer_norm", norm)
    torch.manual_seed(0)
    return MultiHeadAttention(16, 2, dropout=0.4, norm=True), MultiScaleDeformableAttention(16, 2, 2, 2, dropout=0.4, norm=True)


REENTRANT = pytest.mark.parametrize("reentrant", [False, True])


@REENTRANT
def test_without_a_counter_it_is_an_error(operands, reentrant):  # noqa: F811
    drop = Dropout(0.5)
    x = torch.randn(20, 20, requires_grad=True)
    out = checkpoint(drop, x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="counter"):
        out.square().sum().backward()
    assert x.grad is None


@REENTRANT
def test_a_counter_draws_the_same_mask(operands, reentrant):  # noqa: F811
    drop = Dropout(0.5)
    x, r = torch.randn(20, 20, requires_grad=True), torch.randn(20, 20, requires_grad=True)
    counter = drop.next()
    assert int(drop.state[1]) == 1
    out = checkpoint(drop, x, r, counter, use_reentrant=reentrant)
    out.square().sum().backward()
    got = x.grad, r.grad
    x.grad = r.grad = None
    want = drop(x, residual=r, counter=counter)
    want.square().sum().backward()
    assert torch.equal(out, want) and torch.equal(got[0], x.grad) and torch.equal(got[1], r.grad)
    assert int(drop.state[1]) == 1                   # no draw of its own


@REENTRANT
@pytest.mark.parametrize("which", [0, 1])
def test_layers(layers, reentrant, which):
    layer = layers[which]
    query = torch.randn(2, 5, 16, requires_grad=True)
    shapes, starts = torch.tensor([[4, 5], [2, 3]]), torch.tensor([0, 20])
    others = (None, None, None, None) if which == 0 else (torch.rand(2, 5, 2), torch.randn(2, 26, 16), shapes, starts, None)
    drop = layer.dropout if which == 0 else layer.output_dropout
    grads = []
    counter = drop.next()
    for again in (False, True):
        out = checkpoint(layer, query, *others, counter, use_reentrant=reentrant) if again else layer(query, *others, counter=counter)
        grads.append(torch.autograd.grad(out.square().sum(), query) if not reentrant else (out.square().sum().backward(), query.grad)[1:])
        query.grad = None
    assert torch.equal(grads[0][0], grads[1][0])
    out = checkpoint(layer, query, *others, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="counter"):
        out.sum().backward()
    plain = MultiHeadAttention(16, 2) if which == 0 else MultiScaleDeformableAttention(16, 2, 2, 2)
    with pytest.raises(ValueError, match="dropout"):
        plain(query, *others, counter=counter)
    layer.eval()                                     # no draw, whether or not there is a counter
    assert torch.equal(layer(query, *others, counter=counter), layer(query, *others))
    checkpoint(layer, query, *others, use_reentrant=reentrant).sum().backward()


def test_steps_without_recomputation_draw_as_ever(operands):  # noqa: F811
    drop = Dropout(0.5)
    x = torch.randn(9, requires_grad=True)
    for n in range(3):
        drop(x).sum().backward()
        assert int(drop.state[1]) == n + 1
    with torch.no_grad():
        drop(x)
    assert int(drop.state[1]) == 4


def test_another_modules_dropout_in_its_place(layers):
    """A user's replacement, which knows no counter."""
    layer = layers[0].eval()
    x = torch.randn(2, 5, 16)
    want = layer(x)
    layer.dropout = torch.nn.Dropout(0.4).eval()
    assert torch.equal(layer(x), want)
