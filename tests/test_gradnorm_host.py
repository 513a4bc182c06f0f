"""The gradient norm's argument checks, made on the host before any CUDA call."""
import ctypes

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def so():
    from scale_deformable_attention_msda_gb300 import binding, build
    build.build()
    return binding.load()


class Lists:
    """A msda_grad_list_t and the host arrays it points to."""

    def __init__(self, sizes=(256, 0, 7), dtypes=(0, 1, 2), at=None, outs=None, out_dtypes=None, count=None):
        from scale_deformable_attention_msda_gb300.binding import msda_grad_list_t
        n = len(sizes)
        at = at or [FAKE] * n
        self.at = (ctypes.c_void_p * n)(*at)
        self.outs = (ctypes.c_void_p * n)(*(outs or at))
        self.sizes = (ctypes.c_int64 * n)(*sizes)
        self.dtypes = (ctypes.c_int32 * n)(*dtypes)
        self.out_dtypes = (ctypes.c_int32 * n)(*(out_dtypes or dtypes))
        arrays = (self.at, self.outs, self.sizes, self.dtypes, self.out_dtypes)
        self.struct = msda_grad_list_t(n if count is None else count, *[ctypes.addressof(a) for a in arrays])


def norm(so, lists, kind=0, to=FAKE, ws=FAKE, size=1 << 40):
    return so.msda_grad_norm(ctypes.byref(lists.struct) if lists else None, kind, to, ws, size, None)


def clip(so, lists, kind=0, max_norm=1.0, to=FAKE, ws=FAKE, size=1 << 40):
    return so.msda_clip_grad_norm(ctypes.byref(lists.struct) if lists else None, kind, max_norm, to, ws, size, None)


@pytest.mark.parametrize("call", [norm, clip])
def test_errors_before_any_launch(so, call):
    assert call(so, None) == 1
    assert call(so, Lists(count=-1)) == 2
    assert call(so, Lists(sizes=(256, -1, 7))) == 2
    assert call(so, Lists(sizes=(256, 0, (1 << 38) + 1))) == 2
    assert call(so, Lists(dtypes=(0, 9, 2))) == 3
    assert call(so, Lists(dtypes=(0, -1, 2))) == 3
    assert call(so, Lists(), kind=2) == 3
    assert call(so, Lists(at=[FAKE, None, None])) == 1      # the empty one's may be NULL
    assert call(so, Lists(at=[FAKE + 2, FAKE, FAKE])) == 4
    assert call(so, Lists(), to=None) == 1
    assert call(so, Lists(), to=FAKE + 2) == 4
    assert call(so, Lists(dtypes=(0, 3, 2)), to=FAKE + 4) == 4       # a double beside an fp64 tensor
    assert call(so, Lists(), ws=None) == 5
    assert call(so, Lists(), ws=FAKE + 8) == 4
    lists = Lists()
    lists.struct.sizes = None
    assert call(so, lists) == 1


def test_clip_errors(so):
    assert clip(so, Lists(), max_norm=-1.0) == 2
    assert clip(so, Lists(), max_norm=float("nan")) == 2
    assert clip(so, Lists(out_dtypes=(1, 1, 2))) == 3        # fp32 into bf16
    assert clip(so, Lists(out_dtypes=(0, 1, 1))) == 3        # fp16 into bf16
    assert clip(so, Lists(dtypes=(3, 1, 2), out_dtypes=(0, 1, 2))) == 3
    assert clip(so, Lists(outs=[FAKE, FAKE, None])) == 1
    assert clip(so, Lists(outs=[FAKE, FAKE, FAKE + 2], out_dtypes=(0, 1, 0))) == 4
    lists = Lists()
    lists.struct.outs = None
    assert clip(so, lists) == 1


def test_workspace(so):
    def need(lists):
        return so.msda_grad_norm_workspace_bytes(ctypes.byref(lists.struct))
    one = need(Lists(sizes=(5,), dtypes=(0,)))
    assert one > 0 and need(Lists(sizes=(), dtypes=())) == one and need(Lists(sizes=(0,), dtypes=(0,))) == one
    assert need(Lists()) == 2 * one                          # two types with entries
    assert need(Lists(sizes=[3] * 961, dtypes=[1] * 961)) == 2 * one
    assert need(Lists(dtypes=(0, 9, 2))) == 0
    assert norm(so, Lists(), size=2 * one - 1) == 5
    assert clip(so, Lists(), size=2 * one - 1) == 5


def test_binding_refuses_cpu_tensors(so):
    from scale_deformable_attention_msda_gb300 import binding
    with pytest.raises(ValueError, match="CUDA"):
        binding.msda_grad_norm([torch.zeros(3)])
