"""Attention's steps one after another in the same memory: each reads its own statistics,
packed mask and parts, whatever the step before left there."""
import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, make_mask, operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("sizes", [(2, 300, 300, 8, 8, 32), (1, 700, 900, 4, 2, 64), (1, 260, 1500, 2, 1, 128), (2, 100, 1000, 4, 4, 32)], ids=str)
@pytest.mark.parametrize("want", [(1, 1, 1), (1, 0, 0), (0, 1, 1)], ids=str)
def test_steps_in_turn(sizes, want, dt):
    B, Q, S, M = sizes[:4]
    cases = []
    for seed in range(3):
        q, k, v, go, gen = operands(*sizes, dt, seed=100 * seed)
        cases.append((q, k, v, go, make_mask("heads", B, M, Q, S, gen) if seed != 1 else None))

    def step(q, k, v, go, mask):
        out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
        grads = binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, rest=rest, want=want)
        assert [g is not None for g in grads] == [bool(w) for w in want]
        return [out, lse] + [g for g in grads if g is not None]

    alone = []
    for c in cases:
        torch.cuda.synchronize()
        alone.append(step(*c))
        torch.cuda.synchronize()
    full = [binding.msda_attention_backward(c[3], *c[:3], *a[:2], mask=c[4]) for c, a in zip(cases, alone)]
    assert all(torch.isfinite(g).all() for grads in full for g in grads)
    different = 0
    for turn in range(20):
        for c, want_it in zip(cases, alone):
            different += sum((~(a == b)).sum() for a, b in zip(step(*c), want_it))
    assert int(different) == 0
