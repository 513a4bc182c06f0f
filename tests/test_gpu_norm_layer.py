"""The attention layer with its norm, its gradients and their clipping, run
together as a training step runs them, against float64."""
import numpy as np
import pytest
import torch

import oracle
from norm_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding, workloads as wl
from scale_deformable_attention_msda_gb300.layer import LayerNorm, MultiScaleDeformableAttention
from test_gpu_layer import LEVELS, _rel, reference_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    oracle.build()


def setting(given_residual, dtype=torch.float32):
    torch.manual_seed(0)
    B, Q, heads, hd = 2, 40, 2, 32
    dim = heads * hd
    layer = MultiScaleDeformableAttention(dim, heads, len(LEVELS), 3, norm=True)
    with torch.no_grad():
        for p in layer.parameters():
            p.add_(0.05 * torch.randn_like(p))
    S = int(sum(h * w for h, w in LEVELS))
    dev = torch.device("cuda")
    t = {"query": torch.randn(B, Q, dim), "value": torch.randn(B, S, dim),
         "residual": torch.randn(B, Q, dim) if given_residual else None,
         "reference": torch.rand(B, Q, len(LEVELS), 2), "grad": torch.randn(B, Q, dim)}
    t = {k: None if v is None else v.to(dev, dtype) for k, v in t.items()}
    t["shapes"] = torch.tensor(wl.spatial_shapes(LEVELS), device=dev)
    t["starts"] = torch.tensor(wl.level_start_index(LEVELS), device=dev)
    return layer.to(dev, dtype), t


def run(layer, t):
    return layer(t["query"], t["reference"], t["value"], t["shapes"], t["starts"], residual=t["residual"])


@pytest.mark.parametrize("given_residual", [False, True])
def test_a_training_step(given_residual):
    """Forward, backward and clipping at 0.1, in float64 beside it. The bars are those of
    the layer's own test, 1e-4 relative in L2 norm."""
    layer, t = setting(given_residual)
    for k in ("query", "value", "residual"):
        if t[k] is not None:
            t[k].requires_grad_()
    out = run(layer, t)
    out.backward(t["grad"])
    grads = {n: p.grad.clone() for n, p in layer.named_parameters()}
    norm = binding.clip_grad_norm_(layer.parameters(), 0.1)

    r = {k: t[k].detach().double().cpu().requires_grad_() for k in ("query", "value")}
    res = t["residual"].detach().double().cpu().requires_grad_() if given_residual else r["query"]
    attention, P = reference_layer(layer, r["query"], t["reference"].double().cpu(), r["value"],
                                   wl.spatial_shapes(LEVELS), wl.level_start_index(LEVELS))
    s = attention + res
    var, mean = torch.var_mean(s, -1, correction=0, keepdim=True)
    want = (s - mean) / torch.sqrt(var + layer.norm.eps) * P["norm.weight"] + P["norm.bias"]
    want.backward(t["grad"].double().cpu())
    assert _rel(out, want) <= 1e-4
    for k, v in r.items():
        assert _rel(t[k].grad, v.grad) <= 1e-4, k
    if given_residual:
        assert _rel(t["residual"].grad, res.grad) <= 1e-4
    assert set(grads) == set(P)
    for n, p in P.items():
        assert _rel(grads[n], p.grad) <= 1e-4, n
    exact = torch.stack([p.grad.square().sum() for p in P.values()]).sum().sqrt()
    assert abs(float(norm) / float(exact) - 1) <= 1e-4
    factor = 0.1 / (float(norm) + 1e-6)
    for n, p in layer.named_parameters():
        assert _rel(p.grad, grads[n].double() * factor) <= 1e-6, n
    clipped = torch.stack([p.grad.double().square().sum() for p in layer.parameters()]).sum().sqrt()
    assert abs(float(clipped) / 0.1 - 1) <= 1e-4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_layer_in_16_bits(dtype):
    """The norm of what the projection gave, elementwise, and one step's gradients finite."""
    layer, t = setting(False, dtype)
    layer.norm.float()                   # the norm's parameters in float32
    out = run(layer, t)
    seen = {}
    hook = layer.output_proj.register_forward_hook(lambda m, i, o: seen.update(o=o))
    again = run(layer, t)
    hook.remove()
    assert torch.equal(out, again)
    want = reference(seen["o"], layer.norm.weight, layer.norm.bias, t["query"])
    check("out", out, want["out"])
    out.backward(t["grad"])
    assert all(p.grad.isfinite().all() and p.grad.dtype == p.dtype for p in layer.parameters())
    binding.clip_grad_norm_(layer.parameters(), 0.1)       # mixed types


def test_a_captured_training_step():
    """Forward, backward and clipping in one graph, replayed on new inputs."""
    layer, t = setting(True)
    params = list(layer.parameters())
    leaves = [t[k].requires_grad_() for k in ("query", "value", "residual")]

    def step():
        grads = torch.autograd.grad(run(layer, t), leaves + params, t["grad"])
        norm = binding.msda_clip_grad_norm(list(grads[3:]), 0.1)
        return [norm, *grads]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for seed in range(2):
        torch.manual_seed(100 + seed)
        with torch.no_grad():
            for k in ("query", "value", "residual", "grad"):
                t[k].copy_(torch.randn_like(t[k]))
        g.replay()
        torch.cuda.synchronize()
        got = [c.clone() for c in captured]
        want = step()
        torch.cuda.synchronize()
        # grad_value's atomics vary in their order; all else has the same bits
        for a, b in zip(got, want):
            assert _rel(a, b) <= 1e-5


def test_the_plain_layer_is_unchanged():
    torch.manual_seed(3)
    a = MultiScaleDeformableAttention(64, 2, len(LEVELS), 3)
    torch.manual_seed(3)
    b = MultiScaleDeformableAttention(64, 2, len(LEVELS), 3, norm=True)
    assert set(b.state_dict()) - set(a.state_dict()) == {"norm.weight", "norm.bias"}
    assert all(torch.equal(v, b.state_dict()[k]) for k, v in a.state_dict().items())
    layer, t = setting(True)
    layer.norm = None
    with pytest.raises(ValueError, match="residual"):
        run(layer, t)


def test_layer_norm_module():
    torch.manual_seed(0)
    x, r = torch.randn(30, 256, device="cuda"), torch.randn(30, 256, device="cuda")
    m = LayerNorm(256, eps=1e-6).cuda()
    check("out", m(x), reference(x, m.weight, m.bias, None, 1e-6)["out"])
    out, s = m(x, r, return_sum=True)
    want = reference(x, m.weight, m.bias, r, 1e-6)
    check("out", out, want["out"])
    check("sum", s, want["sum"])
    m = LayerNorm(256, bias=False).cuda()
    assert [n for n, _ in m.named_parameters()] == ["weight"]
    check("out", m(x), reference(x, m.weight, None)["out"])
