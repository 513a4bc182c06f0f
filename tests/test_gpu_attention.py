"""Attention, forward and backward, against its definition in float64 with elementwise
bounds (attention_reference.py)."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding, build

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
IDS = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    binding.msda_device_check()
    yield
    assert binding.msda_device_check() == 0          # no wait ran out


def draw(shape, dt, gen, size=1.0):
    return (size * torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float64)).to(dt)


def operands(B, Q, S, M, N, D, dt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7 * Q + S)
    return (draw((B, Q, M, D), dt, gen, 1.3), draw((B, S, N, D), dt, gen, 1.3), draw((B, S, N, D), dt, gen),
            draw((B, Q, M * D), dt, gen, 0.1), gen)


def make_mask(kind, B, M, Q, S, gen):
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=gen)  # noqa: E731
    if kind == "none":
        return None
    if kind == "padding":
        ends = (rand(B) * (S + 1)).long()
        return (torch.arange(S, device="cuda") < ends[:, None])[:, None, None, :]
    if kind == "pairs":
        return rand(Q, S) < 0.6
    if kind == "heads":
        return rand(B, M, Q, S) < 0.5
    if kind == "queries":                            # some queries attend nothing, the others everything
        return (rand(B, 1, Q, 1) < 0.5)
    if kind == "blocks":                             # most tiles are empty or full
        i, j = torch.arange(Q, device="cuda")[:, None], torch.arange(S, device="cuda")[None, :]
        return (i // 128 + j // 128) % 2 == 0
    raise ValueError(kind)


def compare(q, k, v, go, mask=None, scale=None):
    out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, scale=scale, rest=True)
    want = reference(q, k, v, mask, scale, go)
    check("out", out, want["out"])
    check("lse", lse, want["lse"])
    exact = reference(q, k, v, mask, scale, go, exact_out=True)
    eo = exact["out"][0]
    given = eo.to(q.dtype)
    left = None if q.dtype == F32 else (eo - given.double()).to(q.dtype)
    grads = binding.msda_attention_backward(go, q, k, v, given, exact["lse"][0].float(), mask=mask, scale=scale, rest=left)
    for name, grad in zip(("gq", "gk", "gv"), grads):
        check(name, grad, exact[name])
    grads = binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, scale=scale, rest=rest)
    for name, grad in zip(("gq", "gk", "gv"), grads):
        check(name + " after the forward", grad, want[name])


# one token and one key; tiles' first and last rows and columns; every width of the channels
SIZES = [(1, 1, 1, 1, 1, 8), (2, 3, 5, 2, 1, 16), (1, 64, 64, 1, 1, 32), (1, 128, 128, 1, 1, 32), (2, 129, 127, 4, 2, 24),
         (1, 300, 300, 8, 8, 32), (2, 1, 1000, 8, 2, 64), (1, 65, 257, 3, 3, 96), (1, 257, 64, 2, 1, 128), (2, 100, 700, 4, 4, 40),
         (1, 17, 2100, 2, 1, 128), (3, 33, 129, 6, 2, 8), (1, 40, 300, 48, 1, 16), (1, 513, 255, 2, 2, 64), (2, 255, 513, 1, 1, 56),
         (1, 700, 130, 3, 1, 120)]


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_against_float64(sizes, dt):
    q, k, v, go, _ = operands(*sizes, dt)
    compare(q, k, v, go)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("kind", ["padding", "pairs", "heads", "queries", "blocks"])
@pytest.mark.parametrize("sizes", [(2, 5, 9, 2, 1, 16), (2, 130, 200, 4, 2, 32), (1, 300, 300, 2, 2, 64), (3, 70, 900, 2, 1, 128), (2, 1, 1500, 6, 2, 40)], ids=str)
def test_masks(sizes, kind, dt):
    q, k, v, go, gen = operands(*sizes, dt, seed=3)
    B, Q, S, M = sizes[:4]
    compare(q, k, v, go, make_mask(kind, B, M, Q, S, gen))


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_scales(dt):
    q, k, v, go, _ = operands(1, 70, 200, 2, 2, 32, dt)
    for scale in (0.0, 1e-12, 1e-4, 1.0, 3.0):
        compare(q, k, v, go, scale=scale)


@pytest.mark.parametrize("dt", [BF16, F16], ids=IDS)
def test_gradients_of_any_size(dt):
    """Scaled gradients: fp16 operands of the products stay in range."""
    q, k, v, go, _ = operands(1, 150, 200, 2, 1, 32, dt)
    for size in ((1e-3, 30.0) if dt == F16 else (1e-20, 1e10)):
        compare(q, k, v, (go.double() * size).to(dt))


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_large_scores(dt):
    """A few keys have nearly all weight; the maximum rises along the keys."""
    q, k, v, go, _ = operands(1, 140, 600, 2, 2, 64, dt)
    k = (k.double() * torch.linspace(0.2, 4.0, 600, device="cuda")[None, :, None, None]).to(dt)
    compare(q, k, v, go)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_places_hold_anything(dt, bad):
    B, Q, S, M, N, D = 2, 70, 150, 4, 2, 32
    q, k, v, go, gen = operands(B, Q, S, M, N, D, dt)
    on = torch.ones(B, 1, Q, S, dtype=torch.bool, device="cuda")
    on[0, :, :, 100:] = False                        # padded keys
    on[1, :, 7] = False                              # a query without keys
    on[1, :, 20:30, 60] = False                      # one key, for some queries
    compare(q, k, v, go, on)
    k[0, 100:], v[0, 100:] = bad, bad
    q[1, 7], go[1, 7] = bad, bad
    out, lse, rest = binding.msda_attention_forward(q, k, v, mask=on, rest=True)
    want = reference(q, k, v, on, None, go)
    check("out", out, want["out"])
    grads = binding.msda_attention_backward(go, q, k, v, out, lse, mask=on, rest=rest)
    for name, grad in zip(("gq", "gk", "gv"), grads):
        check(name, grad, want[name])
    # a key that some queries must not see: theirs stay finite, the others' do not
    v[1, 60] = bad
    out = binding.attention(q, k, v, mask=on).view(B, Q, M, D)
    sees = on[1, 0, :, 60]
    assert torch.isfinite(out[1, ~sees]).all() and torch.isfinite(out[0]).all()
    assert not torch.isfinite(out[1, sees]).any()


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_layouts(dt):
    """Parts of one projection, other orders of dimensions, odd offsets, repeated batches."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, L, M, N, D = 2, 150, 4, 2, 32
    both = draw((B, L, M + 2 * N, D), dt, gen)
    q, k, v = both.split([M, N, N], 2)
    go = draw((B, L, M * D), dt, gen)
    compare(q, k, v, go)
    compare(q.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(0, 1).contiguous().transpose(0, 1), v, go)
    compare(draw((B, L, D, M), dt, gen).transpose(2, 3), k, v, go)           # channels not contiguous: copied
    shifted = draw((B * L * M * D + 1,), dt, gen)[1:].view(B, L, M, D)       # off a 16-byte boundary: copied
    compare(shifted, k, v, go)
    compare(q, k[:1].expand(B, L, N, D), v[:1].expand(B, L, N, D), go)
    wide = torch.rand(B, 2 * L, 3 * L, device="cuda", generator=gen) < 0.6
    compare(q, k, v, go, wide[:, None, ::2, ::3])
    compare(q, k, v, go, wide[:, None, :L, 1:L + 1])
    compare(q, k, v, go, wide.transpose(1, 2)[:, None, :L, :L])


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_nothing_to_attend(dt):
    for B, Q, S in ((0, 3, 4), (2, 0, 5), (2, 3, 0), (1, 200, 0), (1, 0, 200)):
        q, k, v, go, _ = operands(B, Q, S, 4, 2, 16, dt)
        mask = torch.ones(Q, S, dtype=torch.bool, device="cuda")
        for m in (None, mask):
            out, lse, rest = binding.msda_attention_forward(q, k, v, mask=m, rest=True)
            assert (out == 0).all() and (lse == -float("inf")).all()
            grads = binding.msda_attention_backward(go, q, k, v, out, lse, mask=m, rest=rest)
            for t, g in zip((q, k, v), grads):
                assert g.shape == t.shape and (g == 0).all()


def test_positions_past_32_bits():
    """A cache whose rows lie further apart than 32 bits reach."""
    step, S, D = 1 << 23, 300, 64
    cache = torch.empty(step * S, dtype=BF16, device="cuda")     # 5 GB
    k = cache.as_strided((1, S, 1, D), (step * S, step, D, 1))
    v = cache.as_strided((1, S, 1, D), (step * S, step, D, 1), 1024)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k.copy_(draw(k.shape, BF16, gen))
    v.copy_(draw(v.shape, BF16, gen))
    q, go = draw((1, 9, 2, D), BF16, gen), draw((1, 9, 2 * D), BF16, gen)
    compare(q, k, v, go)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_autograd(dt):
    q, k, v, go, gen = operands(2, 90, 160, 4, 2, 32, dt)
    mask = make_mask("heads", 2, 4, 90, 160, gen)
    want = reference(q, k, v, mask, None, go)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = binding.attention(*leaves, mask=mask)
    check("out", out.detach(), want["out"])
    for name, grad in zip(("gq", "gk", "gv"), torch.autograd.grad(out, leaves, go)):
        check(name, grad, want[name])
    # some of them, a gradient that is not contiguous, keys that repeat
    for wanted in ((0,), (1,), (2,), (0, 2)):
        leaves = [t.clone().requires_grad_(i in wanted) for i, t in enumerate((q, k, v))]
        out = binding.attention(*leaves, mask=mask)
        across = go.transpose(0, 1).contiguous().transpose(0, 1)
        grads = torch.autograd.grad(out, [leaves[i] for i in wanted], across)
        for i, grad in zip(wanted, grads):
            check("gq gk gv".split()[i], grad, want["gq gk gv".split()[i]])
    one = [t.clone().requires_grad_() for t in (q, k[:1], v[:1])]
    out = binding.attention(one[0], one[1].expand_as(k), one[2].expand_as(v), mask=mask)
    shared = reference(q, k[:1].expand_as(k), v[:1].expand_as(v), mask, None, go)
    for i, grad in enumerate(torch.autograd.grad(out, one, go)):
        value, bound = shared["gq gk gv".split()[i]]
        if i:
            value, bound = value.sum(0, keepdim=True), bound.sum(0, keepdim=True) + 2 * value.abs().sum(0, keepdim=True) * 2.0 ** -8
        check("gq gk gv".split()[i], grad, (value, bound))
    with pytest.raises(RuntimeError):                # second derivatives
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        first = torch.autograd.grad(binding.attention(*leaves).sum(), leaves[0], create_graph=True)[0]
        first.sum().backward()


def test_gradients_against_differences():
    q, k, v, go, gen = operands(1, 9, 14, 2, 1, 16, F32)
    mask = make_mask("heads", 1, 2, 9, 14, gen)
    mask[0, 0, 0, 0] = mask[0, 1, 0, 0] = True
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(binding.attention(*leaves, mask=mask), leaves, go)
    for i in range(3):
        for _ in range(4):
            d = torch.randn(leaves[i].shape, device="cuda", generator=gen, dtype=torch.float64)
            moved = []
            for step in (1e-4, -1e-4):               # in float64: the definition's differences
                x = [t.double() for t in (q, k, v)]
                x[i] = x[i] + step * d
                moved.append((reference(*x_as(x), mask)["out"][0] * go.double()).sum())
            slope = float((moved[0] - moved[1]) / 2e-4)
            got = float((grads[i].double() * d).sum())
            size = float((grads[i].double() * d).abs().sum())
            # an fp32 gradient's error of 1e-5 of the terms' sizes, the differences' second order of 1e-7
            assert abs(got - slope) <= 2e-5 * size + 1e-6


def x_as(tensors):
    """float64 tensors as reference() takes them (their type only picks the bounds)."""
    class Held:
        def __init__(self, t):
            self.t, self.dtype, self.shape, self.device = t, F32, t.shape, t.device

        def detach(self):
            return self.t
    return [Held(t) for t in tensors]


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_same_bits(dt):
    """The same call gives the same bits, whatever runs beside it."""
    for sizes, kind in (((2, 333, 700, 6, 2, 64), "heads"), ((2, 500, 300, 4, 4, 32), "none"), ((1, 2, 5000, 8, 2, 128), "padding")):
        q, k, v, go, gen = operands(*sizes, dt)
        mask = make_mask(kind, sizes[0], sizes[3], sizes[1], sizes[2], gen)
        first = None
        noise = torch.randn(2048, 2048, device="cuda")
        side = torch.cuda.Stream()
        for i in range(8):
            with torch.cuda.stream(side):
                for _ in range(i % 3):
                    noise = noise @ noise * 1e-3
            out, lse = binding.msda_attention_forward(q, k, v, mask=mask)
            got = [out, lse, *binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask)]
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_streams_and_graphs(dt):
    """Two captured steps, replayed in turn and on new inputs; a call on another stream."""
    steps = []
    for seed, sizes in ((1, (2, 140, 300, 4, 2, 32)), (2, (1, 1, 4000, 8, 2, 64))):
        q, k, v, go, gen = operands(*sizes, dt, seed=seed)
        mask = make_mask("pairs", 2, 4, sizes[1], sizes[2], gen)

        def call(q=q, k=k, v=v, go=go, mask=mask):
            out, lse = binding.msda_attention_forward(q, k, v, mask=mask)
            return [out, lse, *binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask)]
        call()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            held = call()
        steps.append((graph, held, call, (q, k, v, go)))
    for turn in range(3):
        for graph, held, call, inputs in steps:
            for t in inputs:
                t.copy_(draw(t.shape, dt, torch.Generator(device="cuda").manual_seed(turn)))
        for graph, *_ in steps:
            graph.replay()
        for graph, held, call, _ in steps:
            assert all(torch.equal(a, b) for a, b in zip(held, call()))
    side = torch.cuda.Stream()
    q, k, v, go = steps[0][3]
    torch.cuda.synchronize()
    out, lse = binding.msda_attention_forward(q, k, v, stream=side)
    grads = binding.msda_attention_backward(go, q, k, v, out, lse, stream=side)
    side.synchronize()
    plain, lse2 = binding.msda_attention_forward(q, k, v)
    assert torch.equal(plain, out)
    assert all(torch.equal(a, b) for a, b in zip(grads, binding.msda_attention_backward(go, q, k, v, plain, lse2)))


def test_threads():
    import threading
    cases = [operands(1, 60 + 40 * i, 200 + 90 * i, 4, 2, (32, 64, 128)[i % 3], BF16, seed=i) for i in range(4)]
    want = [binding.attention(*c[:3]) for c in cases]
    got = [[] for _ in cases]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(binding.attention(*cases[i][:3]))
            torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all(torch.equal(w, o) for w, outs in zip(want, got) for o in outs)


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_writes_nothing_else(dt):
    """Outputs given inside larger buffers: what lies around stays."""
    q, k, v, _, _ = operands(1, 133, 190, 3, 3, 40, dt)
    buffer = torch.full((4096 + 133 * 120 + 4096,), 7.0, dtype=dt, device="cuda")
    out = buffer[4096:4096 + 133 * 120].view(1, 133, 120)
    got, _ = binding.msda_attention_forward(q, k, v, out=out)
    assert got is out and (buffer[:4096] == 7).all() and (buffer[-4096:] == 7).all()
    check("out", out, reference(q, k, v)["out"])


def test_refusals():
    q, k, v, go, _ = operands(1, 4, 6, 2, 1, 16, BF16)
    call = binding.attention
    for bad in (lambda: call(q.double(), k.double(), v.double()), lambda: call(q, k.float(), v), lambda: call(q, k, v[:, :5]),
                lambda: call(q[..., :12], k[..., :12], v[..., :12]), lambda: call(q[0], k, v), lambda: call(q[:, :, :1].repeat(1, 1, 3, 1), k.repeat(1, 1, 2, 1), v.repeat(1, 1, 2, 1)),
                lambda: call(q, k, v, mask=torch.zeros(4, 6, device="cuda")), lambda: call(q, k, v, mask=torch.ones(5, 6, dtype=torch.bool, device="cuda")),
                lambda: call(q, k, v, mask=torch.ones(4, 6, dtype=torch.bool)), lambda: call(q, k, v, scale=-1.0), lambda: call(q, k, v, scale=float("nan")),
                lambda: call(q, k.cpu(), v), lambda: binding.msda_attention_forward(q, k, v, out=torch.empty(1, 4, 31, device="cuda", dtype=BF16)),
                lambda: binding.msda_attention_forward(q, k, v, out=q.view(1, 4, 32))):
        with pytest.raises(ValueError):
            bad()
    out, lse = binding.msda_attention_forward(q, k, v)
    with pytest.raises(ValueError):
        binding.msda_attention_backward(go, q, k, v, out, lse.double())
    with pytest.raises(ValueError):
        binding.msda_attention_backward(go[:, :3], q, k, v, out, lse)
    from torch.fx.experimental.proxy_tensor import make_fx
    with pytest.raises(RuntimeError, match="recorded"):
        make_fx(lambda a: binding.attention(a, k, v))(q)


def test_checked_build():
    """The range-checked library gives the same, without a fault."""
    cases = [operands(2, 70, 130, 4, 2, 32, dt) for dt in (F32, BF16, F16)]
    want = [binding.attention(*c[:3]) for c in cases]
    try:
        binding.use_library(build.CHECKED_LIBRARY)
        binding.msda_device_check()
        for c, w in zip(cases, want):
            out, lse = binding.msda_attention_forward(*c[:3])
            assert torch.equal(out, w)
            binding.msda_attention_backward(c[3], *c[:3], out, lse)
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()
