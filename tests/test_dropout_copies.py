"""Dropout's generators in copies of a layer, as a detector's decoder is made of: each draws
masks of its own. On the CPU, the launches replaced by stand-ins."""
import copy
import pickle

import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention, MultiScaleDeformableAttention


@pytest.fixture
def operands(monkeypatch):
    """Draws on the CPU: a mask that is a function of the two words of the counter."""
    def draw(state):
        drawn = state.clone()
        state[1] += 1
        return drawn

    def drop(x, p, counter, residual=None):
        gen = torch.Generator().manual_seed(hash(tuple(counter.tolist())) % 2 ** 62)
        kept = torch.where(torch.rand(x.shape, generator=gen) >= p, x / (1 - p), 0.0)
        return kept if residual is None else residual + kept

    monkeypatch.setattr(binding, "dropout_next", draw)
    monkeypatch.setattr(binding, "dropout", drop)


def seeds(model):
    return [int(m.state[0]) for m in model.modules() if isinstance(m, Dropout)]


def test_copies_have_seeds_of_their_own(operands):
    layer = MultiHeadAttention(32, 4, dropout=0.1)
    other = MultiScaleDeformableAttention(32, 4, dropout=0.1)
    stack = torch.nn.ModuleList([copy.deepcopy(m) for m in (layer, other) for _ in range(6)] + [layer, other])
    assert len(set(seeds(stack))) == 14
    twice = copy.deepcopy(stack)                     # and copies of copies
    assert len(set(seeds(stack) + seeds(twice))) == 28
    assert all(int(m.state[1]) == 0 for m in twice.modules() if isinstance(m, Dropout))


def test_copies_draw_masks_of_their_own(operands):
    x = torch.ones(64, 64)
    first = Dropout(0.5)
    second = copy.deepcopy(first)
    a, b = first(x), second(x)
    share = float((a == b).double().mean())
    assert abs(share - 0.5) < 0.1                    # 4,096 entries: 0.008 of one deviation


def test_a_copy_keeps_all_else(operands):
    class Named(Dropout):
        def __init__(self, p, name):
            super().__init__(p)
            self.name = name

    drop = Named(0.25, ["a"]).eval()
    drop.inner = torch.nn.Linear(2, 2)
    other = copy.deepcopy(drop)
    assert type(other) is Named and other.p == 0.25 and other.name == ["a"] and other.name is not drop.name
    assert not other.training and other.inner is not drop.inner and torch.equal(other.inner.weight, drop.inner.weight)
    shared = [drop, drop]
    a, b = copy.deepcopy(shared)
    assert a is b                                    # one module in two places stays one


def test_what_is_stored_and_loaded_continues(operands):
    drop = Dropout(0.5)
    x = torch.ones(100)
    drop(x)
    loaded, pickled = Dropout(0.5), pickle.loads(pickle.dumps(drop))
    loaded.load_state_dict(drop.state_dict())
    want = drop(x)
    assert torch.equal(loaded(x), want) and torch.equal(pickled(x), want)


def test_the_same_seed_of_torchs_gives_the_same_seeds(operands):
    made = []
    for _ in range(2):
        torch.manual_seed(5)
        layer = MultiHeadAttention(32, 4, dropout=0.1)
        made.append(seeds(torch.nn.ModuleList([layer] + [copy.deepcopy(layer) for _ in range(3)])))
    assert made[0] == made[1]
