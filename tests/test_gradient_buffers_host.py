"""GradientBuffers' hold on its tensors' memory, on the CPU: tensors that say they are on
a GPU, and no launch."""
import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding, build


class Cuda(torch.Tensor):
    is_cuda = True


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def tensors(*sizes):
    return [torch.zeros(n).as_subclass(Cuda) for n in sizes]


def as_if_given_the_same_block(buf):
    """What the buffers know of addresses, as an allocator would have it that gave every
    storage its old one."""
    if hasattr(buf, "_memory"):
        buf._memory = (buf._read_memory()[0], buf._memory[1])
    else:
        buf._addresses = list(map(torch.Tensor.data_ptr, buf._all))


def test_tensors_as_they_were():
    buf = binding.GradientBuffers(tensors(1000, 0, 7), out=tensors(1000, 0, 7))
    before = [list(buf._at), list(buf._out_at)]
    buf._prepare()
    assert [list(buf._at), list(buf._out_at)] == before


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("out", [False, True])
def test_a_storage_made_smaller_at_the_same_address(at, out):
    """An allocator may give a freed block again: the address alone does not show that the
    memory behind a tensor has become less."""
    grads, outs = tensors(1000, 500), tensors(1000, 500)
    buf = binding.GradientBuffers(grads, out=outs if out else None)
    t = (outs if out else grads)[at]
    t.untyped_storage().resize_(0)
    t.untyped_storage().resize_(400)
    as_if_given_the_same_block(buf)
    with pytest.raises(ValueError, match="resized"):
        buf._prepare()


def test_a_storage_made_larger_is_followed():
    grads = tensors(1000, 500)
    buf = binding.GradientBuffers(grads)
    grads[0].untyped_storage().resize_(40000)
    buf._prepare()
    assert grads[0].data_ptr() == buf._at[0]


def test_views_of_one_buffer():
    flat = torch.zeros(1500).as_subclass(Cuda)
    buf = binding.GradientBuffers(list(flat.split([1000, 500])))
    buf._prepare()
    flat.untyped_storage().resize_(4 * 1499)
    as_if_given_the_same_block(buf)
    with pytest.raises(ValueError, match="resized"):
        buf._prepare()
