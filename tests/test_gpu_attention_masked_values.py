"""What lies in masked places does not show in attention's results, finite values among it:
large ones there change no bit, and none of another batch entry's, head's or query's either."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, draw, make_mask, operands  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(2, 70, 150, 4, 2, 32), (1, 300, 300, 3, 3, 64), (2, 40, 1100, 2, 1, 128), (1, 1, 700, 4, 1, 64), (2, 260, 65, 8, 2, 16)]


def step(q, k, v, go, mask=None):
    out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
    return [out, lse, *binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, rest=rest)]


@pytest.mark.parametrize("dt", [F16, BF16, F32], ids=IDS)
@pytest.mark.parametrize("kind", ["padding", "pairs", "heads", "queries", "blocks"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_finite_values(sizes, kind, dt):
    B, Q, S, M, N, D = sizes
    q, k, v, go, gen = operands(*sizes, dt, seed=4)
    mask = make_mask(kind, B, M, Q, S, gen).expand(B, M, Q, S).clone()
    mask[:, :, :, S // 2:S // 2 + 3] = False         # keys that no query attends
    if Q > 20:
        mask[:, :, 11:14] = False                    # queries without keys
    go = go.view(B, Q, M, D)
    keys = mask.view(B, N, M // N, Q, S).any(3).any(2).transpose(1, 2)[..., None]
    queries = mask.any(3).transpose(1, 2)[..., None]
    results = []
    for fill in (0.0, 60000.0, -60000.0):
        dirty = [torch.where(some, t, torch.full_like(t, fill)) for t, some in ((q, queries), (k, keys), (v, keys), (go, queries))]
        results.append(step(*dirty[:3], dirty[3].reshape(B, Q, M * D), mask))
    for other in results[1:]:
        for name, a, b in zip(("out", "lse", "gq", "gk", "gv"), results[0], other):
            assert torch.equal(a, b), name
    clean = [torch.where(some, t, torch.zeros_like(t)) for t, some in ((q, queries), (k, keys), (v, keys), (go, queries))]
    want = reference(*clean[:3], mask, None, clean[3].reshape(B, Q, M * D))
    for name, got in zip(("out", "lse", "gq", "gk", "gv"), results[0]):
        check(name, got, want[name])


@pytest.mark.parametrize("dt", [F16, BF16], ids=IDS)
def test_a_cache_of_large_garbage(dt):
    """Keys behind the sequences' ends: the bounds are those of the keys that are attended."""
    B, Q, S, M, N, D = 2, 50, 4096, 4, 2, 64
    q, k, v, go, _ = operands(B, Q, S, M, N, D, dt, seed=5)
    live = torch.arange(S, device="cuda") < torch.tensor([3300, 801], device="cuda")[:, None]
    mask, live = live[:, None, None, :].expand(B, M, Q, S).clone(), live[:, :, None, None]
    mask[1, :, 5] = False
    go = go.view(B, Q, M, D)
    go[1, 5] = 0.0
    clean = [torch.where(live, t, torch.zeros_like(t)) for t in (k, v)]
    want = reference(q, *clean, mask, None, go.reshape(B, Q, M * D))
    dirty = [torch.where(live, t, torch.full_like(t, 60000.0)) for t in (k, v)]
    go[1, 5] = 60000.0
    for name, got in zip(("out", "lse", "gq", "gk", "gv"), step(q, *dirty, go.reshape(B, Q, M * D), mask)):
        check(name, got, want[name])


@pytest.mark.parametrize("dt", [F16, BF16, F32], ids=IDS)
@pytest.mark.parametrize("sizes", [(2, 130, 200, 4, 2, 32), (2, 300, 100, 4, 4, 64), (2, 33, 500, 2, 2, 128)], ids=str)
def test_one_entry_beside_another(sizes, dt):
    """A batch entry's, and a head's, large gradients and values change nothing in the others."""
    B, Q, S, M, N, D = sizes
    q, k, v, go, _ = operands(*sizes, dt, seed=6)
    go = go.view(B, Q, M, D)
    first = step(q, k, v, go.reshape(B, Q, M * D))
    loud_v, loud_go = v.clone(), go.clone()
    loud_v[1] *= 1024
    loud_go[1] *= 1024
    loud_v[:, :, 1] *= 16
    loud_go[:, :, M // N:2 * (M // N)] *= 16
    second = step(q, k, loud_v, loud_go.reshape(B, Q, M * D))
    for name, a, b in zip(("gq", "gk", "gv"), first[2:], second[2:]):
        heads = M // N if name == "gq" else 1
        assert torch.equal(a[0, :, :heads], b[0, :, :heads]), name


@pytest.mark.parametrize("dt", [F16, BF16, F32], ids=IDS)
def test_one_query_beside_another(dt):
    """A query's gradient keeps its digits beside queries of much larger ones."""
    q, k, v, go, _ = operands(1, 200, 300, 2, 1, 64, dt, seed=7)
    loud = go.clone()
    loud[:, ::2] *= 32768                           # of 0.1 times a normal number
    first, second = step(q, k, v, go), step(q, k, v, loud)
    assert torch.equal(first[2][:, 1::2], second[2][:, 1::2])
