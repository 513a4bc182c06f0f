"""Layer norm's kernels under tracing and forward-mode differentiation."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from norm_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import LayerNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("residual,total", [(False, False), (True, False), (True, True)])
def test_a_traced_module_normalises_its_own_inputs(grad, residual, total):
    torch.manual_seed(0)
    m = LayerNorm(96).cuda()

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.norm = m

        def forward(self, x, *r):
            return self.norm(x, *r, return_sum=total)

    def rows():
        return tuple(torch.randn(7, 96, device="cuda") for _ in range(1 + residual))

    with torch.set_grad_enabled(grad):
        traced = torch.jit.trace(Block(), rows(), check_trace=False)
        for _ in range(3):
            x = rows()
            got = traced(*x)
            want = reference(x[0], m.weight, m.bias, x[1] if residual else None)
            check("out", got[0] if total else got, want["out"])
            if total:
                check("sum", got[1], want["sum"])


def test_a_tangent_is_refused():
    x = torch.randn(3, 8, device="cuda")
    m = LayerNorm(8).cuda().requires_grad_(False)
    with fwAD.dual_level():
        for grad in (False, True):
            with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="jvp"):
                m(fwAD.make_dual(x, torch.ones_like(x)))
        check("out", m(x), reference(x, m.weight, m.bias)["out"])


def test_an_output_given_by_the_caller_advances_its_version():
    """A tensor saved for a backward pass cannot be overwritten unnoticed."""
    x = torch.randn(3, 8, device="cuda")
    leaf = torch.ones(3, 8, device="cuda", requires_grad=True)
    out = torch.ones(3, 8, device="cuda")
    y = (leaf * out).sum()               # saves out
    binding.msda_layer_norm_forward(x, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():         # such tensors have no version
        out = torch.empty(3, 8, device="cuda")
        binding.msda_layer_norm_forward(x, out=out)
    check("out", out, reference(x, None, None)["out"])
