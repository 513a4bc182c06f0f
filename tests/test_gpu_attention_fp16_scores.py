"""Attention's gradients of fp16 data at scores far from ordinary ones: larger than fp16's
largest number, of log-sums as large, and at scales whose inverse fp16 does not hold."""
import pytest
import torch

from test_gpu_attention import BF16, F16, IDS, _lib, compare, draw, make_mask  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(1, 140, 200, 2, 1, 64), (2, 70, 130, 2, 2, 128), (1, 300, 257, 4, 2, 32), (1, 40, 500, 2, 2, 16)]


@pytest.mark.parametrize("dt", [F16, BF16], ids=IDS)
@pytest.mark.parametrize("size,scale", [(130.0, 1.0), (60.0, 8.0), (350.0, 0.125), (2000.0, 1e-6), (12000.0, 3e-9), (12000.0, 1e-11)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_scores_of_any_size(sizes, size, scale, dt):
    """Queries and keys of `size`: the products reach 2^17 to 2^33, the log-sums 2^20 at most. Where
    scores are ordinary after the scale, so are the errors; where they are not, all stays finite
    (the bounds grow with the scores)."""
    B, Q, S, M, N, D = sizes
    gen = torch.Generator(device="cuda").manual_seed(Q)
    q, k = draw((B, Q, M, D), dt, gen, size), draw((B, S, N, D), dt, gen, size)
    v, go = draw((B, S, N, D), dt, gen), draw((B, Q, M * D), dt, gen, 0.1)
    compare(q, k, v, go, scale=scale)
    compare(q, k, v, go, make_mask("heads", B, M, Q, S, gen), scale=scale)


def test_large_differences_of_the_sums():
    """Rows whose gradient's sums (delta) lie far from each other: each keeps its digits."""
    B, Q, S, M, N, D = 1, 200, 300, 2, 1, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = draw((B, Q, M, D), F16, gen), draw((B, S, N, D), F16, gen), draw((B, S, N, D), F16, gen, 200.0)
    go = draw((B, Q, M, D), F16, gen) * torch.logspace(-2, 2, Q, device="cuda").view(1, Q, 1, 1)
    compare(q, k, v, go.to(F16).reshape(B, Q, M * D))
