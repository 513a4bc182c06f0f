"""Attention's forward of a few rows a key head (a decoded token and the query heads that
share its key head), against its definition in float64; and ordinary calls around it:
operands that are one tensor, gradients that repeat one value, parts that need no gradient."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding, build
from test_gpu_attention import BF16, F16, F32, IDS, _lib, compare, make_mask, operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("rows", [(1, 1), (1, 2), (1, 3), (1, 4), (2, 1), (2, 2), (3, 1), (4, 1), (5, 1)], ids=str)
def test_rows(rows, dt):
    """Q queries of G heads a key head, with key lengths around a warp's, a block's and a
    split's share, in channels that fill their lanes and that do not."""
    Q, G = rows
    for S, D in ((1, 8), (7, 32), (33, 40), (255, 64), (513, 128), (2049, 24), (5000, 96)):
        q, k, v, go, _ = operands(3, Q, S, 2 * G, 2, D, dt, seed=S)
        compare(q, k, v, go)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("kind", ["padding", "pairs", "heads", "queries"])
def test_masks_of_few_rows(kind, dt):
    for Q, G, S, D in ((1, 4, 700, 64), (2, 2, 1100, 32), (4, 1, 3001, 128), (1, 1, 90, 16)):
        q, k, v, go, gen = operands(2, Q, S, 2 * G, 2, D, dt, seed=1)
        compare(q, k, v, go, make_mask(kind, 2, 2 * G, Q, S, gen))


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_cache_with_more_room_than_tokens(dt, bad):
    """What lies behind each sequence's end, and in sequences without a token, may be anything."""
    B, S, M, N, D = 4, 1500, 8, 2, 64
    q, k, v, _, _ = operands(B, 1, S, M, N, D, dt, seed=2)
    ends = torch.tensor([0, 1, 700, S], device="cuda")
    live = torch.arange(S, device="cuda") < ends[:, None]
    live = live[:, :, None, None]
    mask = live.permute(0, 2, 3, 1)
    clean, dirty = ([torch.where(live, t, torch.full_like(t, fill)) for t in (k, v)] for fill in (0.0, bad))
    want = reference(q, *clean, mask, None, None)
    out, lse = binding.msda_attention_forward(q, *dirty, mask=mask)
    assert out[0].eq(0).all() and lse[0].eq(-float("inf")).all()
    check("out", out, want["out"])
    check("lse", lse, want["lse"])


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_large_scores_of_a_few_rows(dt):
    """The maximum rises, and falls, along the keys."""
    q, k, v, go, _ = operands(2, 1, 3000, 4, 1, 64, dt, seed=3)
    for lo, hi in ((0.2, 4.0), (4.0, 0.2)):
        grown = (k.double() * torch.linspace(lo, hi, 3000, device="cuda")[None, :, None, None]).to(dt)
        compare(q, grown, v, go)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_one_tensor_in_two_places(dt):
    """Keys that are the values, and queries that are both: the gradients are added, in an
    order of the engine's."""
    q, k, _, go, _ = operands(2, 40, 40, 4, 4, 32, dt, seed=4)
    for a, b in ((q, k), (q, q)):
        x, y = a.clone().requires_grad_(), b.clone().requires_grad_()
        if a is b:
            y = x
        binding.attention(x, y, y).backward(go)
        gq, gk, gv = parts = [t.clone().requires_grad_() for t in (a, b, b)]
        binding.attention(*parts).backward(go)
        gq, gk, gv = gq.grad, gk.grad, gv.grad
        if a is b:
            assert any(torch.equal(x.grad, sum_) for sum_ in ((gq + gk) + gv, (gq + gv) + gk, (gk + gv) + gq))
        else:
            assert torch.equal(x.grad, gq) and torch.equal(y.grad, gk + gv)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_gradients_that_repeat(dt):
    """The gradient of a sum is one value at strides of zero."""
    q, k, v, _, _ = operands(1, 30, 50, 2, 2, 32, dt, seed=5)
    grads = []
    for ones in (False, True):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        out = binding.attention(*leaves)
        out.backward(torch.ones_like(out)) if ones else out.sum().backward()
        grads.append([t.grad for t in leaves])
    for x, y in zip(*grads):
        assert torch.equal(x, y)


@pytest.mark.parametrize("needs", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (0, 0, 0)], ids=str)
def test_gradients_that_are_wanted(needs):
    q, k, v, go, _ = operands(1, 30, 50, 2, 1, 32, BF16, seed=6)
    full = [t.clone().requires_grad_() for t in (q, k, v)]
    binding.attention(*full).backward(go)
    some = [t.clone().requires_grad_(bool(n)) for t, n in zip((q, k, v), needs)]
    out = binding.attention(*some)
    assert out.requires_grad == any(needs)
    if any(needs):
        out.backward(go)
    for n, s, f in zip(needs, some, full):
        assert torch.equal(s.grad, f.grad) if n else s.grad is None


def test_second_derivatives_are_refused():
    q, k, v, go, _ = operands(1, 5, 6, 1, 1, 16, F32, seed=7)
    q.requires_grad_()
    grad, = torch.autograd.grad(binding.attention(q, k, v), q, go, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()


def test_checked_build_of_few_rows():
    """The range-checked library, with few rows, split keys and masks: no fault."""
    try:
        binding.use_library(build.CHECKED_LIBRARY)
        binding.msda_device_check()
        for sizes, dt in (((2, 1, 1500, 4, 2, 40), F32), ((2, 1, 1500, 4, 2, 40), F16), ((1, 3, 700, 2, 2, 128), F32), ((2, 90, 900, 4, 2, 64), BF16)):
            q, k, v, go, gen = operands(*sizes, dt, seed=8)
            compare(q, k, v, go, make_mask("heads", sizes[0], sizes[3], sizes[1], sizes[2], gen))
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()
