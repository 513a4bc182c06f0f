"""Attention of few queries over many keys, whose gradients are computed by blocks of their
own kind: sizes on both sides of where these begin, masks, and what lies in masked places."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, compare, make_mask, operands  # noqa: F401

pytestmark = pytest.mark.gpu

# key tiles of 128: 480, 512, 472, 461, 464; then 456, and queries too many
SIZES = [(4, 20, 3800, 4, 4, 32), (8, 3, 2000, 8, 4, 64), (2, 100, 15000, 4, 2, 24), (1, 120, 59000, 2, 1, 64), (4, 1, 3700, 16, 4, 16),
         (4, 64, 3640, 8, 4, 32), (4, 257, 3800, 4, 4, 32)]


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("kind", ["none", "padding", "heads", "blocks"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_against_float64(sizes, kind, dt):
    B, Q, S, M, N, D = sizes
    q, k, v, go, gen = operands(*sizes, dt)
    compare(q, k, v, go, make_mask(kind, B, M, Q, S, gen))


@pytest.mark.parametrize("dt", [BF16, F16], ids=IDS)
@pytest.mark.parametrize("fill", [60000.0, float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", SIZES[:3] + SIZES[4:5], ids=str)
def test_masked_places(sizes, fill, dt):
    B, Q, S, M, N, D = sizes
    q, k, v, go, gen = operands(*sizes, dt, seed=1)
    mask = make_mask("heads", B, M, Q, S, gen)
    mask[..., 1000:1003] = False                     # keys that no query attends
    mask[..., S - 70:] = False
    clean = [k.clone(), v.clone()]
    for t in clean:
        t[:, 1000:1003] = 0.0
        t[:, S - 70:] = 0.0
    want = reference(q, *clean, mask, None, go)
    dirty = [t.clone() for t in clean]
    for t in dirty:
        t[:, 1000:1003] = fill
        t[:, S - 70:] = fill
    if Q > 2:
        go = go.clone().view(B, Q, M, D)
        mask[:, :, 1] = False
        go[:, 1] = 0.0
        want = reference(q, *clean, mask, None, go.view(B, Q, M * D))
        go[:, 1] = fill
        go = go.view(B, Q, M * D)
    out, lse, rest = binding.msda_attention_forward(q, *dirty, mask=mask, rest=True)
    got = [out, lse, *binding.msda_attention_backward(go, q, *dirty, out, lse, mask=mask, rest=rest)]
    for name, g in zip(("out", "lse", "gq", "gk", "gv"), got):
        check(name, g, want[name])


@pytest.mark.parametrize("dt", [BF16, F16], ids=IDS)
@pytest.mark.parametrize("size,scale", [(130.0, 1.0), (60.0, 8.0), (12000.0, 3e-9)])
def test_scores_of_any_size(size, scale, dt):
    q, k, v, go, _ = operands(4, 40, 3800, 4, 4, 64, dt, seed=2)
    q, k = (t.double().mul(size / 1.3).clamp(-6e4, 6e4).to(dt) for t in (q, k))
    compare(q, k, v, go, scale=scale)


def test_steps_in_turn():
    """Both launches of a backward, one step after another in the same memory."""
    cases = []
    for seed in range(3):
        q, k, v, go, gen = operands(4, 100, 4000, 8, 8, 32, BF16, seed=100 * seed)
        cases.append((q, k, v, go, make_mask("heads", 4, 8, 100, 4000, gen) if seed != 1 else None))

    def step(q, k, v, go, mask):
        out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
        return [out, lse, *binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, rest=rest)]
    alone = []
    for c in cases:
        torch.cuda.synchronize()
        alone.append(step(*c))
        torch.cuda.synchronize()
    different = sum((~(a == b)).sum() for _ in range(15) for c, w in zip(cases, alone) for a, b in zip(step(*c), w))
    assert int(different) == 0
