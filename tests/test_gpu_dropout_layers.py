"""Layers with dropout on the GPU: copies of one layer, layers run again for their backward,
and generators that are moved, stored and captured."""
import copy

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention, MultiScaleDeformableAttention
from test_gpu_dropout import _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def layer_and_operands(which):
    torch.manual_seed(which)
    query = torch.randn(2, 60, 64, device="cuda", requires_grad=True)
    if which == 0:
        return MultiHeadAttention(64, 4, dropout=0.3, norm=True).cuda(), query, ()
    layer = MultiScaleDeformableAttention(64, 4, 2, 4, dropout=0.3, norm=True).cuda()
    return layer, query, (torch.rand(2, 60, 2, device="cuda"), torch.randn(2, 26, 64, device="cuda"),
                          torch.tensor([[4, 5], [2, 3]], device="cuda"), torch.tensor([0, 20], device="cuda"))


@pytest.mark.parametrize("reentrant", [False, True])
@pytest.mark.parametrize("which", [0, 1])
def test_recomputed_layers(which, reentrant):
    layer, query, others = layer_and_operands(which)
    drop = layer.dropout if which == 0 else layer.output_dropout
    counter = drop.next()
    grads = []
    for again in (False, True):
        out = checkpoint(layer, query, *others, counter=counter, use_reentrant=False) if again and not reentrant else \
            checkpoint(lambda q: layer(q, *others, counter=counter), query, use_reentrant=True) if again else layer(query, *others, counter=counter)
        out.square().sum().backward()
        grads.append([out.detach(), query.grad] + [p.grad for p in layer.parameters()])
        query.grad = None
        layer.zero_grad()
    # the deformable layer's gradients are added by atomics, in an order that changes
    for a, b in zip(*grads):
        assert torch.equal(a, b) if which == 0 else torch.allclose(a, b, rtol=1e-4, atol=1e-4 * float(a.abs().max()))
    out = checkpoint(layer, query, *others, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="counter"):
        out.square().sum().backward()
    torch.cuda.synchronize()


def test_a_decoder_of_copies():
    layer = MultiHeadAttention(64, 4, dropout=0.5).cuda()
    layers = [copy.deepcopy(layer) for _ in range(6)]
    ones = torch.ones(128, 64, device="cuda")
    masks = [m.dropout(ones) != 0 for m in layers + [layer]]
    for i, a in enumerate(masks):
        for b in masks[:i]:
            assert abs(float((a == b).double().mean()) - 0.5) < 0.05        # 8,192 entries: 9 deviations
    assert all(m.dropout.state.is_cuda for m in layers)


def test_a_generator_is_moved_and_stored():
    drop = Dropout(0.5)
    words = drop.state.tolist()
    drop = drop.to("cuda").half()
    assert drop.state.is_cuda and drop.state.tolist() == words
    x = torch.ones(1000, device="cuda")
    drop(x)
    stored = drop.cpu().state_dict()
    assert stored["state"].tolist() == [words[0], 1]
    other = Dropout(0.5).cuda()
    held = other.state.data_ptr()
    graph = torch.cuda.CUDAGraph()
    other(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = other(x)
    other.load_state_dict(stored)                    # the captured step reads the same two words
    assert other.state.data_ptr() == held
    graph.replay()
    assert torch.equal(out, binding.dropout(x, 0.5, torch.tensor([words[0], 1], device="cuda")))
    other.reseed(77)
    graph.replay()
    assert torch.equal(out, binding.dropout(x, 0.5, torch.tensor([77, 0], device="cuda")))
