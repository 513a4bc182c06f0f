"""An infinite entry of the output's gradient: the values' gradients are not finite in its
channel, and what they are in the others."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("sizes", [(1, 200, 260, 2, 1, 64), (2, 300, 140, 2, 2, 32), (1, 150, 300, 4, 1, 128), (1, 40, 90, 2, 2, 16)], ids=str)
def test_values_gradients_in_the_other_channels(sizes, bad, dt):
    B, Q, S, M, N, D = sizes
    q, k, v, go, _ = operands(*sizes, dt)
    go.view(B, Q, M, D)[0, 17, 0, 3] = 0.0
    want = reference(q, k, v, None, None, go)
    out, lse, rest = binding.msda_attention_forward(q, k, v, rest=True)
    go.view(B, Q, M, D)[0, 17, 0, 3] = bad
    gq, gk, gv = binding.msda_attention_backward(go, q, k, v, out, lse, rest=rest)
    touched = torch.zeros_like(gv, dtype=torch.bool)
    touched[0, :, 0, 3] = True
    assert torch.equal(~torch.isfinite(gv), touched)
    value, bound = want["gv"]
    check("gv", torch.where(touched, value.to(dt), gv), (value, bound + value.abs() * touched))
    # the query's own gradient, and all keys' of its head, are those of an infinite slope
    assert not torch.isfinite(gq[0, 17, 0]).any() and not torch.isfinite(gk[0, :, 0]).any()
    at = torch.ones(Q, dtype=torch.bool, device="cuda")
    at[17] = False
    value, bound = want["gq"]
    check("gq", gq[:, at], (value[:, at], bound[:, at]))
    check("gk", gk[1:], tuple(t[1:] for t in want["gk"]))
