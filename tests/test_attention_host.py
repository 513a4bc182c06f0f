"""Attention's and dropout's argument checks, made on the host before any CUDA call."""
import ctypes

import pytest
import torch

FAKE = 0x10000   # aligned; no call below reaches a launch


@pytest.fixture(scope="module")
def so():
    from scale_deformable_attention_msda_gb300 import binding, build
    build.build()
    return binding.load()


def dims(B=2, Q=300, S=400, M=8, N=4, D=32, **strides):
    from scale_deformable_attention_msda_gb300.binding import msda_attention_dims_t
    three = ctypes.c_int64 * 3
    return msda_attention_dims_t(B, Q, S, M, N, D, three(*strides.get("q", (Q * M * D, M * D, D))), three(*strides.get("k", (S * N * D, N * D, D))),
                                 three(*strides.get("v", (S * N * D, N * D, D))), (ctypes.c_int64 * 4)(*strides.get("mask", (0, 0, S, 1))))


def ref(d):
    return ctypes.byref(d) if d is not None else None


def fwd(so, d, dtype=1, q=FAKE, k=FAKE, v=FAKE, mask=None, out=FAKE, rest=None, lse=FAKE, scale=0.1, ws=FAKE, size=1 << 45):
    return so.msda_attention_forward(q, k, v, mask, out, rest, lse, scale, ws, size, ref(d), dtype, None)


def bwd(so, d, dtype=1, q=FAKE, k=FAKE, v=FAKE, mask=None, out=FAKE, rest=None, lse=FAKE, scale=0.1, ws=FAKE, size=1 << 45, go=FAKE,
        gq=FAKE, gk=FAKE, gv=FAKE):
    return so.msda_attention_backward(go, q, k, v, mask, out, rest, lse, gq, gk, gv, scale, ws, size, ref(d), dtype, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_errors_before_any_launch(so, call):
    assert call(so, None) == 1
    for dtype in (3, 9, -1):
        assert call(so, dims(), dtype=dtype) == 3
    for bad in (dict(B=-1), dict(Q=-1), dict(S=-1), dict(Q=(1 << 30) + 1), dict(S=(1 << 30) + 1), dict(N=0), dict(M=7), dict(M=2, N=4), dict(M=1 << 17, N=1),
                dict(D=0), dict(D=4), dict(D=12), dict(D=136), dict(B=1 << 40)):
        assert call(so, dims(**bad)) == 2, bad
    assert call(so, dims(q=(300 * 256, 0, 32))) == 2
    assert call(so, dims(k=(1 << 50, 128, 32))) == 2
    assert call(so, dims(v=(400 * 128, -128, 32))) == 2
    assert call(so, dims(q=(300 * 256, 257, 32))) == 4
    assert call(so, dims(mask=(0, 0, -1, 1)), mask=FAKE) == 2
    for scale in (-0.1, float("nan"), float("inf")):
        assert call(so, dims(), scale=scale) == 2
    for name in ("q", "k", "v", "out"):
        assert call(so, dims(), **{name: None}) == 1
        assert call(so, dims(), **{name: FAKE + 8}) == 4
    assert call(so, dims(), rest=FAKE + 8) == 4
    assert call(so, dims(), lse=FAKE + 2) == 4
    assert call(so, dims(), mask=FAKE, size=16) == 5
    assert call(so, dims(), mask=FAKE, ws=None) == 5
    assert call(so, dims(), mask=FAKE, ws=FAKE + 8) == 4


def test_backward_errors(so):
    assert bwd(so, dims(), gk=None) == 1
    assert bwd(so, dims(), go=None) == 1
    assert bwd(so, dims(), lse=None) == 1
    assert bwd(so, dims(), gv=FAKE + 4) == 4
    assert bwd(so, dims(), ws=None) == 5


def test_nothing_to_do(so):
    assert fwd(so, dims(B=0), q=None, out=None) == 0
    assert fwd(so, dims(Q=0), q=None, out=None) == 0
    assert bwd(so, dims(), gq=None, gk=None, gv=None, q=None) == 0
    assert bwd(so, dims(B=0), q=None) == 0


def test_strides_of_single_entries_are_not_read(so):
    # reaches the workspace check only when all before it passed
    assert bwd(so, dims(B=1, q=(-5, 256, 32), k=(3, 128, 32), v=(0, 128, 32)), ws=None) == 5


def test_workspaces(so):
    for dtype in (0, 1, 2):
        for Q, S in ((1, 1), (300, 300), (1, 16384), (100, 16384), (5000, 5000)):
            d = dims(Q=Q, S=S)
            plain, masked = (so.msda_attention_forward_workspace_bytes(ref(d), dtype, m) for m in (0, 1))
            assert masked >= plain + Q * S // 8              # bits
            back = so.msda_attention_backward_workspace_bytes(ref(d), dtype, 0)
            assert back >= 8 * 2 * 8 * Q                     # two numbers a query and head
            # the splits' parts: at most 64 times the output, and only where few tiles fill the machine
            assert plain <= 64 * 4 * 2 * Q * 8 * 34 + 4096
    assert so.msda_attention_forward_workspace_bytes(ref(dims(D=12)), 1, 0) == 0
    assert so.msda_attention_backward_workspace_bytes(ref(dims()), 7, 0) == 0
    assert so.msda_attention_forward_workspace_bytes(None, 1, 0) == 0


def test_dropout_errors(so):
    def call(x=FAKE, res=None, out=FAKE, n=100, p=0.1, counter=FAKE, dtype=1):
        return so.msda_dropout(x, res, out, n, p, counter, dtype, None)
    assert call(dtype=9) == 3
    assert call(n=-1) == 2 and call(n=(1 << 60) + 1) == 2
    for p in (-0.1, 1.0001, float("nan")):
        assert call(p=p) == 2
    assert call(x=None) == 1 and call(out=None) == 1 and call(counter=None) == 1
    assert call(x=FAKE + 1) == 4 and call(res=FAKE + 1) == 4 and call(out=FAKE + 2, dtype=0) == 4 and call(counter=FAKE + 4) == 4
    assert call(n=0, x=None, out=None, counter=None) == 0
    assert so.msda_dropout_next(None, FAKE, None) == 1 and so.msda_dropout_next(FAKE, None, None) == 1
    assert so.msda_dropout_next(FAKE + 4, FAKE, None) == 4


def test_binding_refuses_cpu_tensors(so):
    from scale_deformable_attention_msda_gb300 import binding
    q = torch.zeros(1, 3, 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.attention(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        binding.msda_attention_forward(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        binding.dropout(torch.zeros(3), 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        binding.dropout_next(torch.zeros(2, dtype=torch.int64))


def test_wait_status_has_a_name(so):
    from scale_deformable_attention_msda_gb300 import binding
    assert b"ran out" in so.msda_status_string(binding.MSDA_ERR_DEVICE_WAIT)
    assert binding.STATUS[binding.MSDA_ERR_DEVICE_WAIT] == "MSDA_ERR_DEVICE_WAIT"
