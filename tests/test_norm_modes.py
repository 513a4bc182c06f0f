"""Layer norm and the gradient norm under torch's modes that do not see a launch on
addresses: forward-mode differentiation, tracing and recording. On the CPU, with the launch
replaced by one that normalises through addresses as the kernels do."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from scale_deformable_attention_msda_gb300 import binding


def values(t):
    """t's entries by their address: nothing that torch could record."""
    return (ctypes.c_float * t.numel()).from_address(t.data_ptr())


@pytest.fixture
def launches(monkeypatch):
    """The CPU's layer norm of rows without parameters in the launch's place; counts calls."""
    count = []

    def forward(x, weight, bias, residual, eps, return_sum, stats, out, pdt, index):
        count.append(1)
        out = torch.empty_like(x) if out is None else out
        C = x.shape[-1]
        stats = torch.empty(2 * (x.numel() // C)) if stats else None
        v, o = values(x), values(out)
        for i in range(x.numel() // C):
            row = v[i * C:(i + 1) * C]
            mean = sum(row) / C
            rstd = (sum((e - mean) ** 2 for e in row) / C + eps) ** -0.5
            for c in range(C):
                o[i * C + c] = (row[c] - mean) * rstd
        return out, None, stats

    monkeypatch.setattr(binding, "_norm_operands", lambda *a, **k: -1)
    monkeypatch.setattr(binding, "_elsewhere", lambda *a, **k: False)
    monkeypatch.setattr(binding, "_norm_forward", forward)
    return count


def test_the_stand_in(launches):
    x = torch.randn(3, 8)
    assert torch.allclose(binding.layer_norm(x), torch.nn.functional.layer_norm(x, (8,)), atol=1e-5)
    assert len(launches) == 1


@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(launches, grad):
    """A tangent is never dropped: an error, whether or not the primal requires grad."""
    x = torch.randn(3, 8, requires_grad=grad)
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones(3, 8))
        with pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
            binding.layer_norm(dual)
        with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
            binding.layer_norm(dual)
        # what carries no tangent is computed as ever
        plain = torch.randn(3, 8)
        assert torch.allclose(binding.layer_norm(plain), torch.nn.functional.layer_norm(plain, (8,)), atol=1e-5)


@pytest.mark.parametrize("grad", [False, True])
def test_a_trace_calls_the_operator(launches, grad):
    x = torch.randn(3, 8)
    with torch.set_grad_enabled(grad):
        traced = torch.jit.trace(lambda t: binding.layer_norm(t) * 2, (x.clone().requires_grad_(grad),), check_trace=False)
        for _ in range(3):
            other = torch.randn(3, 8)
            before = len(launches)
            got = traced(other)
            assert len(launches) == before + 1
            assert torch.allclose(got, 2 * torch.nn.functional.layer_norm(other, (8,)), atol=1e-5)


def test_recording_by_dispatch_is_refused(launches):
    from torch.fx.experimental.proxy_tensor import make_fx
    x = torch.randn(3, 8)
    with pytest.raises(RuntimeError, match="record"):
        make_fx(lambda t: binding.layer_norm(t))(x)
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="record"):
        make_fx(lambda t: binding.layer_norm(t))(leaf)


CALLS = {
    "msda_layer_norm_forward": lambda t: binding.msda_layer_norm_forward(t)[0],
    "msda_layer_norm_backward": lambda t: binding.msda_layer_norm_backward(t, t, t[:, 0], t[:, 0])[0],
    "msda_grad_norm": lambda t: binding.msda_grad_norm([t]),
    "msda_clip_grad_norm": lambda t: binding.msda_clip_grad_norm([t], 1.0),
    "clip_grad_norm_": lambda t: binding.clip_grad_norm_(Holder(t), 1.0),
}


class Holder(list):
    """A parameter whose gradient is t, in a list."""

    def __init__(self, t):
        p = torch.nn.Parameter(torch.zeros(3, 8))
        p.grad = t
        super().__init__([p])


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_addresses_refuse_to_be_recorded(name):
    """They have no node that a trace or a tangent could pass through."""
    from torch.fx.experimental.proxy_tensor import make_fx
    x = torch.randn(3, 8)
    with pytest.raises(RuntimeError, match="record"):
        torch.jit.trace(CALLS[name], (x,), check_trace=False)
    with pytest.raises(RuntimeError, match="record"):
        make_fx(CALLS[name])(x)
    with fwAD.dual_level():
        with pytest.raises(RuntimeError, match="forward"):
            CALLS[name](fwAD.make_dual(x, torch.ones(3, 8)))
