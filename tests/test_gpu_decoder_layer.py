"""A decoder layer's two attention sublayers as they are used together: queries among
themselves with a mask, dropout, norm, deformable attention over a feature map, dropout,
norm; one training step of it against the same in float64."""
import copy

import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding
from scale_deformable_attention_msda_gb300.layer import Dropout, MultiHeadAttention, MultiScaleDeformableAttention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def plain_attention(layer, query, key, value, mask, residual, keep):
    """The sublayer from its definition in float64, its dropout's mask given."""
    proj = lambda p, x: x @ p.weight.double().T + p.bias.double()  # noqa: E731
    B, Q, C = query.shape
    split = lambda x, h: x.view(B, -1, h, layer.head_dim).transpose(1, 2)  # noqa: E731
    q, k, v = split(proj(layer.query_proj, query), layer.num_heads), split(proj(layer.key_proj, key), layer.kv_heads), split(proj(layer.value_proj, value), layer.kv_heads)
    k, v = (t.repeat_interleave(layer.num_heads // layer.kv_heads, 1) for t in (k, v))
    s = q @ k.mT * layer.head_dim ** -0.5
    p = torch.softmax(s.masked_fill(~mask, -float("inf")), -1)
    out = proj(layer.output_proj, (p @ v).transpose(1, 2).reshape(B, Q, C)) * keep + residual
    mean, var = out.mean(-1, keepdim=True), out.var(-1, unbiased=False, keepdim=True)
    return (out - mean) * (var + 1e-5).rsqrt() * layer.norm.weight.double() + layer.norm.bias.double()


@pytest.mark.parametrize("kv_heads", [8, 2])
def test_self_attention_step(kv_heads):
    torch.manual_seed(0)
    layer = MultiHeadAttention(256, 8, kv_heads=kv_heads, dropout=0.1, norm=True).cuda()
    B, Q = 2, 220
    x = torch.randn(B, Q, 256, device="cuda", requires_grad=True)
    pos = torch.randn(B, Q, 256, device="cuda", requires_grad=True)
    group = torch.arange(Q, device="cuda") // 40
    mask = (group[:, None] == group[None, :]) | (group[None, :] == group.max())
    go = torch.randn(B, Q, 256, device="cuda")
    counter = layer.dropout.state.clone()
    out = layer(x + pos, value=x, mask=mask, residual=x)
    leaves = [x, pos] + list(layer.parameters())
    grads = torch.autograd.grad(out, leaves, go)
    keep = binding.dropout(torch.ones(B, Q, 256, device="cuda", dtype=torch.float64), 0.1, counter)
    xd, pd = x.detach().double().requires_grad_(), pos.detach().double().requires_grad_()
    double = copy.deepcopy(layer).double()
    want = plain_attention(double, xd + pd, xd + pd, xd, mask, xd, keep)
    wanted = torch.autograd.grad(want, [xd, pd] + list(double.parameters()), go.double())
    # sums of some 1e3 products of order one in fp32, whose roundings add up like a random walk:
    # 1e3 ** 0.5 * 2 ** -24, four products deep, with a margin of eight
    tol = 8 * 4 * 1000 ** 0.5 * 2.0 ** -24
    assert float((out.double() - want).norm() / want.norm()) <= tol
    for (name, _), got, ref in zip([("x", 0), ("pos", 0)] + list(layer.named_parameters()), grads, wanted):
        # the key's bias moves all scores of a query alike: its gradient is zero up to roundings
        size = ref.norm() if name != "key_proj.bias" else wanted[2 + [n for n, _ in layer.named_parameters()].index("query_proj.bias")].norm()
        assert float((got.double() - ref).norm() / size) <= tol, name


def decoder(dropout):
    torch.manual_seed(1)
    first = MultiHeadAttention(256, 8, dropout=dropout, norm=True).cuda()
    second = MultiScaleDeformableAttention(256, 8, 2, 4, norm=True, dropout=dropout).cuda()
    shapes = torch.tensor([[20, 30], [10, 15]], device="cuda")
    starts = torch.tensor([0, 600], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    query = torch.randn(2, 100, 256, device="cuda", generator=gen)
    memory = torch.randn(2, 750, 256, device="cuda", generator=gen)
    reference = torch.rand(2, 100, 2, device="cuda", generator=gen)

    def run():
        hidden = first(query, mask=None)
        return second(hidden, reference, memory, shapes, starts)
    return first, second, run


def test_layer_with_and_without_dropout():
    first, second, run = decoder(0.1)
    numbers = lambda: [int(first.dropout.state[1]), int(second.output_dropout.state[1])]  # noqa: E731
    a, b = run(), run()
    assert numbers() == [2, 2] and not torch.equal(a, b)
    first.eval(), second.eval()
    a, b = run(), run()
    assert torch.equal(a, b) and numbers() == [2, 2]
    plain_first, plain_second, plain = decoder(0.0)
    plain_first.load_state_dict(first.state_dict(), strict=False)
    plain_second.load_state_dict(second.state_dict(), strict=False)
    assert torch.equal(plain(), a)
    assert not any("dropout" in k for k in plain_second.state_dict())


def test_captured_training_step():
    """Forward, backward and an update in one graph: replays draw anew and keep training finite."""
    first, second, run = decoder(0.2)
    params = list(first.parameters()) + list(second.parameters())

    def step():
        loss = run().square().mean()
        for p, g in zip(params, torch.autograd.grad(loss, params)):
            p.data.add_(g, alpha=-1e-3)
        return loss
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loss = step()
    before = [p.detach().clone() for p in params]
    start = int(first.dropout.state[1])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert int(first.dropout.state[1]) == start + 3
    assert torch.isfinite(loss) and all(torch.isfinite(p).all() for p in params)
    assert any(not torch.equal(p, q) for p, q in zip(params, before))


def test_autocast():
    first, second, run = decoder(0.1)
    first.eval(), second.eval()
    want = run()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        got = first(torch.randn(2, 9, 256, device="cuda"), mask=None)
        assert torch.isfinite(got).all()
    drop = Dropout(0.5).cuda()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        x = torch.randn(4, 256, device="cuda") @ torch.randn(256, 256, device="cuda")
        out = drop(x, residual=torch.randn(4, 256, device="cuda"))
    assert out.dtype == torch.float32 and torch.isfinite(want).all()


def test_refusals():
    with pytest.raises(ValueError):
        MultiHeadAttention(256, 7)
    with pytest.raises(ValueError):
        MultiHeadAttention(256, 8, kv_heads=3)
    with pytest.raises(ValueError):
        MultiHeadAttention(64, 4).cuda()(torch.zeros(1, 2, 64, device="cuda"), residual=torch.zeros(1, 2, 64, device="cuda"))
