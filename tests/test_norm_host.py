"""Layer norm's argument checks, made on the host before any CUDA call."""
import ctypes

import pytest
import torch

FAKE = 0x10000   # aligned; no call below reaches a launch


@pytest.fixture(scope="module")
def so():
    from scale_deformable_attention_msda_gb300 import binding, build
    build.build()
    return binding.load()


def dims(N=600, C=256):
    from scale_deformable_attention_msda_gb300.binding import msda_norm_dims_t
    return msda_norm_dims_t(N, C)


def fwd(so, d, dtype=1, pdt=1, eps=1e-5, x=FAKE, res=FAKE, w=FAKE, b=FAKE, out=FAKE, total=FAKE,
        mean=FAKE, rstd=FAKE):
    return so.msda_layer_norm_forward(x, res, w, b, out, total, mean, rstd, eps,
                                      ctypes.byref(d) if d is not None else None, dtype, pdt, None)


def bwd(so, d, dtype=1, pdt=1, dy=FAKE, x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, gx=FAKE, gw=FAKE, gb=FAKE,
        ws=FAKE, size=1 << 40):
    return so.msda_layer_norm_backward(dy, None, x, None, w, mean, rstd, gx, gw, gb, ws, size,
                                       ctypes.byref(d) if d is not None else None, dtype, pdt, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_errors_before_any_launch(so, call):
    assert call(so, None) == 1
    assert call(so, dims(), dtype=9) == 3
    assert call(so, dims(), dtype=0, pdt=1) == 3            # 16-bit parameters with fp32 data
    assert call(so, dims(), dtype=1, pdt=2) == 3
    assert call(so, dims(), dtype=3, pdt=0) == 3
    assert call(so, dims(C=0)) == 2
    assert call(so, dims(C=(1 << 20) + 1)) == 2
    assert call(so, dims(N=-1)) == 2
    assert call(so, dims(N=1 << 60, C=2)) == 2
    assert call(so, dims(), x=None) == 1
    assert call(so, dims(), x=FAKE + 1) == 4
    assert call(so, dims(), w=FAKE + 2, pdt=0) == 4
    assert call(so, dims(), mean=FAKE + 2) == 4


def test_forward_errors(so):
    assert fwd(so, dims(), out=None) == 1
    assert fwd(so, dims(), mean=None) == 1
    assert fwd(so, dims(), eps=-1e-9) == 2
    assert fwd(so, dims(), eps=float("nan")) == 2
    assert fwd(so, dims(N=0), x=None, out=None) == 0        # empty: nothing launched


def test_backward_workspace(so):
    for dtype in (0, 1, 2, 3):
        for C in (1, 7, 256, 777, 4096, 70001):
            sizes = [so.msda_layer_norm_backward_workspace_bytes(ctypes.byref(dims(N, C)), dtype)
                     for N in (0, 1, 600, 10 ** 6)]
            assert sizes == sorted(sizes) and sizes[0] >= 2 * C * (8 if dtype == 3 else 4)
            # bounded by the blocks of the machine, not by the rows
            assert sizes[-1] <= 152 * 6 * 2 * C * (8 if dtype == 3 else 4)
    need = so.msda_layer_norm_backward_workspace_bytes(ctypes.byref(dims()), 1)
    assert bwd(so, dims(), size=need - 1) == 5
    assert bwd(so, dims(), ws=None) == 5
    assert bwd(so, dims(), ws=FAKE + 8) == 4
    assert so.msda_layer_norm_backward_workspace_bytes(ctypes.byref(dims(C=0)), 1) == 0
    assert so.msda_layer_norm_backward_workspace_bytes(ctypes.byref(dims()), 7) == 0
    assert bwd(so, dims(), gx=None, gw=None, gb=None, x=None) == 0      # nothing asked
    assert bwd(so, dims(N=0), gw=None, gb=None, x=None, ws=None) == 0   # nothing to write


def test_binding_refuses_cpu_tensors(so):
    from scale_deformable_attention_msda_gb300 import binding
    with pytest.raises(ValueError, match="CUDA"):
        binding.layer_norm(torch.zeros(3, 8))
