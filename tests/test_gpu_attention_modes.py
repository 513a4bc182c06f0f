"""Attention's and dropout's kernels under tracing and forward-mode differentiation."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention
from test_gpu_attention import BF16, F32, IDS, _lib, operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dt", [F32, BF16], ids=IDS)
def test_a_trace_attends_its_own_inputs(dt, grad):
    mask = torch.rand(30, 50, device="cuda") < 0.7
    with torch.set_grad_enabled(grad):
        traced = torch.jit.trace(lambda q, k, v, m: binding.attention(q, k, v, mask=m), (*operands(2, 30, 50, 4, 2, 32, dt)[:3], mask), check_trace=False)
        for seed in (1, 2, 3):
            q, k, v, *_ = operands(2, 30, 50, 4, 2, 32, dt, seed=seed)
            check("out", traced(q, k, v, mask), reference(q, k, v, mask)["out"])


@pytest.mark.parametrize("grad", [False, True])
def test_a_traced_layer(grad):
    torch.manual_seed(0)
    layer = MultiHeadAttention(64, 4, norm=True).cuda()
    x = [torch.randn(2, 20, 64, device="cuda") for _ in range(3)]
    with torch.set_grad_enabled(grad):
        traced = torch.jit.trace(layer, (x[0],), check_trace=False)
        for other in x:
            assert torch.equal(traced(other), layer(other))


def test_a_traced_dropout():
    c = torch.tensor([3, 4], device="cuda")
    traced = torch.jit.trace(lambda x, c: binding.dropout(x, 0.5, c), (torch.randn(50, device="cuda"), c), check_trace=False)
    for n in range(3):
        x, c = torch.randn(50, device="cuda"), torch.tensor([3, n], device="cuda")
        assert torch.equal(traced(x, c), binding.dropout(x, 0.5, c))
    with pytest.raises(RuntimeError, match="record"):            # its draws would be one draw
        torch.jit.trace(Dropout(0.5).cuda(), (x,), check_trace=False)


def test_a_tangent_is_refused():
    q, k, v, *_ = operands(1, 5, 6, 2, 1, 16, F32)
    c = torch.tensor([3, 4], device="cuda")
    with fwAD.dual_level():
        for grad in (False, True):
            with torch.set_grad_enabled(grad):
                with pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
                    binding.attention(fwAD.make_dual(q, torch.ones_like(q)), k, v)
                with pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
                    binding.dropout(fwAD.make_dual(q, torch.ones_like(q)), 0.5, c)
        check("out", binding.attention(q, k, v), reference(q, k, v)["out"])
