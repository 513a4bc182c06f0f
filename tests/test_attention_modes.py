"""Attention and dropout under torch's modes that do not see a launch on addresses:
forward-mode differentiation, tracing and recording. On the CPU, the launches replaced by ones
that work through addresses as the kernels do."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from scale_deformable_attention_msda_gb300 import binding


def values(t):
    """t's entries by their address: nothing that torch could record."""
    return (ctypes.c_float * t.numel()).from_address(t.data_ptr())


class Plan:
    default_scale = 1.0


@pytest.fixture
def launches(monkeypatch):
    """In place of the launches: attention that adds up q, k and v, dropout that doubles."""
    count = []

    def attend(q, k, v, mask, plan, index, scale, lse, rest, out):
        count.append(1)
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2] * q.shape[3])
        for o, *x in zip(range(out.numel()), values(q), values(k), values(v)):
            values(out)[o] = sum(x)
        return out, torch.empty(1) if lse else None, None

    def drop(x, p, counter, residual, out):
        count.append(1)
        out = torch.empty_like(x)
        for i, e in enumerate(values(x)):
            values(out)[i] = 2 * e
        return out

    monkeypatch.setattr(binding, "_plan_of", lambda *a: (Plan, -1))
    monkeypatch.setattr(binding, "_elsewhere", lambda *a, **k: False)
    monkeypatch.setattr(binding, "_attend", attend)
    monkeypatch.setattr(binding, "_drop_operands", lambda *a: -1)
    monkeypatch.setattr(binding, "_drop", drop)
    return count


COUNTER = torch.zeros(2, dtype=torch.int64)
CALLS = {"attention": (lambda t: binding.attention(t, t * 1, t * 1), lambda t: (3 * t).flatten(2)),
         "dropout": (lambda t: binding.dropout(t, 0.5, COUNTER), lambda t: 2 * t)}


def operand(grad=False):
    return torch.randn(2, 3, 2, 8, requires_grad=grad)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(launches, name, grad):
    """A tangent is never dropped: an error, whether or not the primal requires grad."""
    call, want = CALLS[name]
    with fwAD.dual_level():
        dual = fwAD.make_dual(operand(grad), torch.ones(2, 3, 2, 8))
        with pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
            call(dual)
        with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError), match="jvp|forward"):
            call(dual)
        plain = operand()                # what carries no tangent is computed as ever
        assert torch.allclose(call(plain), want(plain))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("grad", [False, True])
def test_a_trace_calls_the_operator(launches, name, grad):
    call, want = CALLS[name]
    with torch.set_grad_enabled(grad):
        traced = torch.jit.trace(lambda t: call(t) * 2, (operand().requires_grad_(grad),), check_trace=False)
        for _ in range(3):
            other = operand()
            before = len(launches)
            got = traced(other)
            assert len(launches) == before + 1
            assert torch.allclose(got, 2 * want(other))


@pytest.mark.parametrize("name", CALLS)
def test_recording_by_dispatch_is_refused(launches, name):
    from torch.fx.experimental.proxy_tensor import make_fx
    for leaf in (operand(), operand(True)):
        with pytest.raises(RuntimeError, match="record"):
            make_fx(CALLS[name][0])(leaf)


PLAIN = {"msda_attention_forward": lambda t: binding.msda_attention_forward(t, t, t)[0],
         "msda_attention_backward": lambda t: binding.msda_attention_backward(t, t, t, t, t, t)[0],
         "msda_dropout": lambda t: binding.msda_dropout(t, 0.1, COUNTER)}


@pytest.mark.parametrize("name", PLAIN)
def test_calls_on_addresses_refuse_to_be_recorded(name):
    from torch.fx.experimental.proxy_tensor import make_fx
    x = operand()
    with pytest.raises(RuntimeError, match="record"):
        torch.jit.trace(PLAIN[name], (x,), check_trace=False)
    with pytest.raises(RuntimeError, match="record"):
        make_fx(PLAIN[name])(x)
    with fwAD.dual_level():
        with pytest.raises(RuntimeError, match="forward"):
            PLAIN[name](fwAD.make_dual(x, torch.ones_like(x)))
