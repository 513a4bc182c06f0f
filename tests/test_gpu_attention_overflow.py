"""Scores past fp32's range: never an answer that looks like one of a query without keys."""
import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, draw  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("sizes", [(1, 70, 90, 2, 2, 64), (2, 1, 3000, 4, 1, 32), (1, 300, 200, 2, 1, 128)], ids=str)
@pytest.mark.parametrize("masked", [False, True])
def test_products_that_overflow(sizes, masked, dt):
    B, Q, S, M, N, D = sizes
    gen = torch.Generator(device="cuda").manual_seed(1)
    size, scale = (1e3, 2e38) if dt == F16 else (1e15, 1e20)
    q, k, v = draw((B, Q, M, D), dt, gen, size), draw((B, S, N, D), dt, gen, size), draw((B, S, N, D), dt, gen)
    mask = torch.rand(Q, S, device="cuda", generator=gen) < 0.8 if masked else None
    out, lse = binding.msda_attention_forward(q, k, v, mask=mask, scale=scale)
    # the key of the largest score has all weight
    s = torch.einsum("bqngd,bknd->bngqk", q.double().view(B, Q, N, M // N, D), k.double())
    if masked:
        s = s.masked_fill(~mask, -float("inf"))
    best = s.argmax(-1).flatten(1, 2)                # (B, M, Q)
    heads = torch.arange(M, device="cuda")[:, None] // (M // N)
    want = v[torch.arange(B, device="cuda")[:, None, None], best, heads].transpose(1, 2).reshape(B, Q, M * D)
    right = (out == want).view(B, Q, M, D).all(-1)
    lost = torch.isnan(out).view(B, Q, M, D).all(-1)
    assert (right | lost).all()
    assert not torch.isfinite(lse).any() and not (lse == -float("inf")).any()


def test_scales_past_the_range_are_refused():
    q = torch.ones(1, 2, 1, 16, device="cuda")
    for scale in (2.5e38, 3e38, float("inf")):
        with pytest.raises(ValueError, match="scale"):
            binding.attention(q, q, q, scale=scale)
    assert torch.isfinite(binding.attention(q * 1e-30, q * 1e-30, q, scale=2.3e38)).all()
