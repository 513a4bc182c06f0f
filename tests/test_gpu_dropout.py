"""Dropout: the generator's words against Philox4x32-10 on the host, results against their
definition, gradients, states, refusals."""
import numpy
import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding, build
from scale_deformable_attention_msda_gb300.layer import Dropout

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16, torch.float64]
IDS = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def philox(block, key):
    """Four 32-bit words of four counter words and two key words (Salmon et al., SC 2011)."""
    c, k = list(block), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def halves(n, seed, number, first=0):
    """The 16 bits of entries first to first + n - 1."""
    seed, number, out = seed % 2 ** 64, number % 2 ** 64, []
    for block in range(first // 8, (first + n + 7) // 8):
        words = philox([block & 0xFFFFFFFF, block >> 32, number & 0xFFFFFFFF, number >> 32], [seed & 0xFFFFFFFF, seed >> 32])
        out += [h for w in words for h in (w & 0xFFFF, w >> 16)]
    return numpy.array(out)[first % 8:first % 8 + n]


def test_published_words():
    """The known answers of the method's paper's test vectors."""
    assert philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def counter(seed, number):
    return torch.tensor([seed, number], device="cuda")


def definition(x, p, seed, number, residual=None):
    t = round(p * 65536)
    keep = torch.from_numpy(halves(x.numel(), seed, number) >= t).to(x.device).view(x.shape)
    factor = torch.tensor(65536 / (65536 - t) if t < 65536 else 0.0, dtype=torch.float64 if x.dtype == torch.float64 else torch.float32).item()
    kept = torch.where(keep, x.double() * factor, 0.0)
    return kept if residual is None else kept + residual.double()


def close(got, want, dt):
    half = {torch.float64: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dt]
    inner = 2.0 ** -52 if dt == torch.float64 else 2.0 ** -23     # the product's and the sum's roundings before the last
    tiny = {torch.float16: 2.0 ** -25}.get(dt, 1e-40)
    assert ((got.double() - want).abs() <= (half + 2 * inner) * want.abs() * 1.01 + inner * 16 + tiny).all() if dt in (torch.float32, torch.float64) \
        else ((got.double() - want).abs() <= (half * want.abs() + 2.0 ** -20) * 1.01 + tiny).all()


SHAPES = [(1,), (7,), (8,), (9,), (3, 5), (33, 77), (600, 256), (2, 3, 1031)]


@pytest.mark.parametrize("dt", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("res", [False, True])
def test_definition(shape, dt, res):
    gen = torch.Generator(device="cuda").manual_seed(len(shape) + shape[0])
    x = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float64).to(dt)
    r = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float64).to(dt) if res else None
    for p, seed, number in ((0.1, 5, 0), (0.5, -(2 ** 62) - 3, 2 ** 33 + 1), (0.0, 1, 1), (1.0, 1, 2), (1e-6, 9, -1)):
        out = binding.dropout(x, p, counter(seed, number), residual=r)
        want = definition(x, p, seed, number, r)
        if r is None:
            assert torch.equal(out == 0, want.to(dt) == 0)
        close(out, want, dt)


@pytest.mark.parametrize("dt", TYPES, ids=IDS)
def test_any_alignment(dt):
    """Entries have the same bits wherever the tensors start; what lies around stays."""
    n, c = 1003, counter(3, 4)
    x = torch.randn(n, device="cuda").to(dt)
    want = binding.dropout(x, 0.3, c)
    for off in (1, 2, 3):
        held = torch.full((n + 16,), 7.0, dtype=dt, device="cuda")
        src = torch.zeros(n + 16, dtype=dt, device="cuda")
        src[off:off + n] = x
        binding.msda_dropout(src[off:off + n], 0.3, c, out=held[off + 1:off + 1 + n])
        assert torch.equal(held[off + 1:off + 1 + n], want)
        assert (held[:off + 1] == 7).all() and (held[off + 1 + n:] == 7).all()


def test_entries_past_32_bits():
    """The last entries of a tensor of more than 2^32, and blocks of the generator past 2^29."""
    n = 2 ** 32 + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = binding.msda_dropout(x, 0.25, counter(11, 12), out=x)
    for first in (0, 2 ** 31 - 8, 2 ** 32 - 16, n - 1027):
        many = min(1027, n - first)
        keep = torch.from_numpy(halves(many, 11, 12, first) >= 16384)
        assert torch.equal((out[first:first + many] != 0).cpu(), keep)


@pytest.mark.parametrize("dt", TYPES, ids=IDS)
def test_gradients(dt):
    x = torch.randn(41, 130, device="cuda").to(dt).requires_grad_()
    r = torch.randn(41, 130, device="cuda").to(dt).requires_grad_()
    g = torch.randn(130, 41, device="cuda").to(dt).t()               # not contiguous
    c = counter(7, 8)
    gx, gr = torch.autograd.grad(binding.dropout(x, 0.4, c, residual=r), (x, r), g)
    assert torch.equal(gr, g)
    close(gx, definition(g, 0.4, 7, 8), dt)
    only, = torch.autograd.grad(binding.dropout(x, 0.4, c, residual=r), (r,), g)
    assert torch.equal(only, g)
    only, = torch.autograd.grad(binding.dropout(x, 0.4, c), (x,), g)
    assert torch.equal(only, gx)
    # linear in x: differences are exact products
    e = torch.zeros_like(x)
    e[3, 5] = 1.0
    a = binding.dropout(e.detach(), 0.4, c)
    back = torch.zeros(41, 130, device="cuda", dtype=dt)
    back[3, 5] = 1.0
    gx, = torch.autograd.grad(binding.dropout(x, 0.4, c), (x,), back)
    assert torch.equal(a, gx)
    with pytest.raises(RuntimeError):
        first = torch.autograd.grad(binding.dropout(x, 0.4, c).square().sum(), x, create_graph=True)[0]
        first.sum().backward()


def test_dropped_entries_hold_anything():
    x = torch.ones(4096, device="cuda")
    out = binding.dropout(x, 0.5, counter(1, 1))
    x[out == 0] = float("nan")
    assert torch.equal(binding.dropout(x, 0.5, counter(1, 1)), out)
    x[:] = float("inf")
    r = torch.randn(4096, device="cuda")
    assert torch.equal(binding.dropout(x, 0.5, counter(1, 1), residual=r)[out == 0], r[out == 0])


def test_in_place():
    x, r = torch.randn(5000, device="cuda"), torch.randn(5000, device="cuda")
    want = binding.dropout(x, 0.2, counter(2, 3), residual=r)
    for into in (x.clone(), r.clone()):
        a, b = (into, r) if torch.equal(into, x) else (x, into)
        version = into._version
        assert torch.equal(binding.msda_dropout(a, 0.2, counter(2, 3), residual=b, out=into), want)
        assert into._version > version


def test_share_kept():
    """The share of kept entries is within 6 deviations of 1 - p, also along rows, and two draws differ."""
    n = 1 << 22
    x = torch.ones(1 << 11, 1 << 11, device="cuda")
    for p in (0.05, 0.5, 0.9):
        t = round(p * 65536) / 65536
        kept = binding.dropout(x, p, counter(123, 0)) != 0
        other = binding.dropout(x, p, counter(123, 1)) != 0
        for k in (kept, other):
            assert abs(float(k.double().mean()) - (1 - t)) <= 6 * (t * (1 - t) / n) ** 0.5
        both = (kept & other).double().mean()
        assert abs(float(both) - (1 - t) ** 2) <= 6 * ((1 - t) ** 2 * (1 - (1 - t) ** 2) / n) ** 0.5
        rows = kept.double().mean(1)
        assert float((rows - (1 - t)).abs().max()) <= 6 * (t * (1 - t) / (1 << 11)) ** 0.5


def test_next_draw():
    state = counter(5, 40)
    drawn = [binding.dropout_next(state) for _ in range(3)]
    assert [d.tolist() for d in drawn] == [[5, 40], [5, 41], [5, 42]] and state.tolist() == [5, 43]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    several = [binding.dropout_next(state, stream=streams[i % 4]) for i in range(40)]
    torch.cuda.synchronize()
    assert sorted(d[1].item() for d in several) == list(range(43, 83)) and state[1].item() == 83


def test_module():
    torch.manual_seed(3)
    drop = Dropout(0.3).cuda()
    x, r = torch.randn(50, 70, device="cuda", requires_grad=True), torch.randn(50, 70, device="cuda")
    start = drop.state.clone()
    a, b = drop(x), drop(x, residual=r)
    assert torch.equal(a, binding.dropout(x, 0.3, start)) and drop.state[1] == start[1] + 2
    start[1] += 1
    assert torch.equal(b, binding.dropout(x, 0.3, start, residual=r))
    gx, = torch.autograd.grad(b.sum(), x)
    assert torch.equal(gx != 0, (b - r) != 0) or float(((gx != 0) != ((b - r) != 0)).double().mean()) < 1e-3   # x of a kept entry may vanish beside r
    drop.eval()
    assert drop(x) is x and torch.equal(drop(x, residual=r), r + x)
    again = Dropout(0.3).cuda()
    again.load_state_dict(drop.state_dict())
    assert torch.equal(again(x), binding.dropout(x, 0.3, drop.state))
    with pytest.raises(ValueError):
        Dropout(1.5)


def test_replayed_step_draws_anew():
    drop = Dropout(0.5).cuda()
    x = torch.ones(3000, device="cuda")
    drop(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = drop(x)
    seen = []
    for _ in range(3):
        start = drop.state.clone()
        graph.replay()
        assert torch.equal(out, binding.dropout(x, 0.5, start))
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_refusals():
    x, c = torch.randn(16, device="cuda"), counter(1, 2)
    for bad in (lambda: binding.dropout(x, -0.1, c), lambda: binding.dropout(x, 1.1, c), lambda: binding.dropout(x, float("nan"), c),
                lambda: binding.dropout(x, 0.1, c.cpu()), lambda: binding.dropout(x, 0.1, c.int()), lambda: binding.dropout(x, 0.1, counter(1, 2)[:1]),
                lambda: binding.dropout(x, 0.1, c, residual=x[:8]), lambda: binding.dropout(x, 0.1, c, residual=x.half()),
                lambda: binding.dropout(x.int(), 0.1, c), lambda: binding.msda_dropout(x[:8], 0.1, c, out=x[4:12])):
        with pytest.raises(ValueError):
            bad()
    assert binding.dropout(x[:0], 0.1, c).numel() == 0


def test_checked_build():
    x, c = torch.randn(999, device="cuda"), counter(1, 2)
    want = binding.dropout(x, 0.1, c)
    try:
        binding.use_library(build.CHECKED_LIBRARY)
        binding.msda_device_check()
        assert torch.equal(binding.dropout(x, 0.1, c), want)
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()
