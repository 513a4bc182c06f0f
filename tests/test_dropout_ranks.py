"""Dropout's generators under data parallelism: what synchronises a model's buffers leaves
them alone. Two ranks on the CPU (gloo); and their place in a model's state."""
import os
import socket
import subprocess
import sys

import pytest
import torch

from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention

RANK = """
import sys
import torch
import torch.distributed as dist
from torch import nn
sys.path.insert(0, sys.argv[3])
from scale_deformable_attention_msda_gb300.layer import MultiHeadAttention

class Model(nn.Module):
    def __init__(self):
        super().__init__()
        self.layer = MultiHeadAttention(16, 2, dropout=0.1)
        self.linear = nn.Linear(4, 4)
        self.register_buffer("shared", torch.full((2,), float(rank)))

    def forward(self, x):
        return self.linear(x)

rank = int(sys.argv[1])
dist.init_process_group("gloo", init_method="tcp://127.0.0.1:" + sys.argv[2], rank=rank, world_size=2)
torch.manual_seed(100 + rank)
model = nn.parallel.DistributedDataParallel(Model(), find_unused_parameters=True)
for _ in range(2):
    model(torch.ones(3, 4)).sum().backward()
state = model.module.layer.dropout.state
state[1] += 5 * rank
model(torch.ones(3, 4))
assert model.module.shared.tolist() == [0.0, 0.0]        # a buffer is rank 0's
both = [torch.empty_like(state) for _ in range(2)]
dist.all_gather(both, state)
assert both[0][0] != both[1][0] and both[1][1] - both[0][1] == 5, both
# the same seed of torch's on both ranks: a seed of each one's own
torch.manual_seed(7)
drop = MultiHeadAttention(16, 2, dropout=0.1).dropout
drop.reseed(1000 + rank)
assert drop.state.tolist() == [1000 + rank, 0]
dist.destroy_process_group()
"""


def test_two_ranks(tmp_path):
    script = tmp_path / "rank.py"
    script.write_text(RANK)
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    ranks = [subprocess.Popen([sys.executable, str(script), str(r), str(port), root], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for r in range(2)]
    outs = [r.communicate(timeout=120)[0] for r in ranks]
    assert all(r.returncode == 0 for r in ranks), outs


def test_seeds_that_are_given():
    a, b = Dropout(0.1), Dropout(0.1)
    a.state[1] = 9
    at = a.state.data_ptr()
    a.reseed(-5)
    assert a.state.tolist() == [-5, 0] and a.state.data_ptr() == at
    b.reseed(2 ** 63 + 1)                            # any 64 bits
    assert b.state.tolist() == [1 - 2 ** 63, 0]
    torch.manual_seed(1)
    a.reseed()
    torch.manual_seed(1)
    b.reseed()
    assert torch.equal(a.state, b.state)


def test_the_state_is_stored_and_moved_with_the_model():
    layer = MultiHeadAttention(16, 2, dropout=0.1)
    assert "dropout.state" in layer.state_dict()
    assert not any(t is layer.dropout.state for t in layer.buffers())
    assert layer.half().dropout.state.dtype == torch.int64 and layer.to("meta").dropout.state.is_meta
    layer, other = MultiHeadAttention(16, 2, dropout=0.1), MultiHeadAttention(16, 2, dropout=0.1)
    held = other.dropout.state
    layer.dropout.state[1] = 3
    assert not other.load_state_dict(layer.state_dict()).missing_keys
    assert torch.equal(held, layer.dropout.state) and other.dropout.state is held
    assert layer.state_dict()["dropout.state"].data_ptr() == layer.dropout.state.data_ptr()
    less = {k: v for k, v in layer.state_dict().items() if k != "dropout.state"}
    with pytest.raises(RuntimeError, match="dropout.state"):
        other.load_state_dict(less)
    assert other.load_state_dict(less, strict=False).missing_keys == ["dropout.state"]
    with pytest.raises(RuntimeError, match="dropout.state"):
        other.load_state_dict(dict(layer.state_dict(), **{"dropout.state": torch.zeros(3, dtype=torch.int64)}))
    with pytest.raises(RuntimeError, match="dropout.other"):
        other.load_state_dict(dict(layer.state_dict(), **{"dropout.other": torch.zeros(3)}))
    with torch.device("meta"):
        empty = MultiHeadAttention(16, 2, dropout=0.1)
    empty.load_state_dict(layer.state_dict(), assign=True)
    assert torch.equal(empty.dropout.state, layer.dropout.state)


def test_modules_pickled_with_a_buffer():
    """States of before: the words were among the module's buffers."""
    drop = Dropout(0.1)
    state = dict(drop.__dict__)
    words = state.pop("state", None)
    state["_buffers"] = {"state": drop.state if words is None else words}
    again = Dropout.__new__(Dropout)
    again.__setstate__(state)
    assert not list(again.buffers()) and torch.equal(again.state, drop.state) and list(again.state_dict()) == ["state"]
