"""The attention layer with its norm, and the norm alone, under autocast with a float32
residual stream, as mixed-precision training runs them."""
import pytest
import torch

from norm_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import LayerNorm
from test_gpu_norm_layer import run, setting

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("given_residual", [False, True])
def test_the_layer(dtype, given_residual):
    """The norm takes the projection's 16-bit output and the float32 residual, unrounded, and
    gives float32, as torch's own does; the same layer without the norm gives that
    projection. Gradients: those of the norm elementwise, of the rest present and finite."""
    layer, t = setting(given_residual)
    for k in ("query", "value", "residual"):
        if t[k] is not None:
            t[k].requires_grad_()
    seen = {}

    def keep(module, args, out):
        seen["out"] = out
        out.register_hook(lambda g: seen.update(grad=g))

    hook = layer.output_proj.register_forward_hook(keep)
    with torch.autocast("cuda", dtype=dtype):
        out = run(layer, t)
    hook.remove()
    assert seen["out"].dtype == dtype and out.dtype == torch.float32
    residual = t["residual"] if given_residual else t["query"]
    want = reference(seen["out"].float(), layer.norm.weight, layer.norm.bias, residual, grad_out=t["grad"])
    check("out", out, want["out"])
    out.backward(t["grad"])
    # the gradient of the 16-bit summand is rounded to its type
    value, bound = want["grad_x"]
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    check("grad of the projection", seen["grad"], (value, bound + half * (value.abs() + bound) + 2.0 ** -25))
    check("grad_weight", layer.norm.weight.grad, want["grad_weight"])
    check("grad_bias", layer.norm.bias.grad, want["grad_bias"])
    if given_residual:
        check("grad_x", t["residual"].grad, want["grad_x"])
    for k in ("query", "value"):
        assert t[k].grad.dtype == torch.float32 and t[k].grad.isfinite().all()
    for p in layer.parameters():
        assert p.grad.dtype == p.dtype and p.grad.isfinite().all()
    binding.clip_grad_norm_(layer.parameters(), 0.1)


@pytest.mark.parametrize("types", [(torch.bfloat16, torch.float32), (torch.float32, torch.float16),
                                   (torch.bfloat16, torch.float16)], ids=str)
@pytest.mark.parametrize("params", [torch.float32, torch.bfloat16], ids=str)
def test_the_norm_alone(types, params):
    """Summands of two types are added in the type that holds both, whatever the parameters'."""
    torch.manual_seed(1)
    x, r = (torch.randn(30, 256, device="cuda").to(d) for d in types)
    m = LayerNorm(256).cuda()
    with torch.no_grad():
        m.weight.add_(0.3 * torch.randn_like(m.weight))
        m.bias.add_(torch.randn_like(m.bias))
    m.to(params)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        out, s = m(x, r, return_sum=True)
    want = reference(x.float(), m.weight.float(), m.bias.float(), r.float())
    check("out", out, want["out"])
    check("sum", s, want["sum"])
    out.sum().backward()
    assert m.weight.grad.dtype == params and m.bias.grad.dtype == params
    # outside autocast types are the caller's to agree on
    with pytest.raises(ValueError, match="expected|parameters"):
        m(x, r)


def test_what_agrees_is_left_as_it_is():
    """Autocast changes nothing where both summands have one type."""
    x, r = (torch.randn(30, 256, device="cuda").bfloat16() for _ in range(2))
    m = LayerNorm(256).cuda()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        out = m(x, r)
    assert out.dtype == torch.bfloat16 and torch.equal(out, m(x, r))
