"""Layer norm with a residual, forward and backward, against its definition in
float64 with elementwise bounds (norm_reference.py)."""
import pytest
import torch

from norm_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding, build

pytestmark = pytest.mark.gpu

F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F64, F64)]
IDS = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def operands(N, C, dt, pdt, residual=True, seed=0, offset=0):
    """x, weight, bias, residual, grad_out, grad_sum; `offset`: elements from a 16-byte boundary."""
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + 7 * N + C)

    def rows(scale, shift=0.0):
        flat = torch.randn(N * C + offset, device="cuda", generator=gen, dtype=torch.float64)
        return (flat * scale + shift).to(dt)[offset:].view(N, C)

    w = (1 + 0.3 * torch.randn(C + offset, device="cuda", generator=gen, dtype=torch.float64)).to(pdt)[offset:]
    b = torch.randn(C + offset, device="cuda", generator=gen, dtype=torch.float64).to(pdt)[offset:]
    return (rows(2.0, 0.5), w, b, rows(1.0, -0.2) if residual else None, rows(0.1), rows(0.1))


def run(x, w, b, r, dy, ds, total, eps=1e-5):
    out, s, mean, rstd = binding.msda_layer_norm_forward(x, w, b, r, eps, total)
    grads = binding.msda_layer_norm_backward(dy, x, mean, rstd, w, r, ds if total else None)
    return out, s, *grads


def compare(x, w, b, r, dy, ds, total, eps=1e-5):
    out, s, gx, gw, gb = run(x, w, b, r, dy, ds, total, eps)
    want = reference(x, w, b, r, eps, dy, ds if total else None)
    check("out", out, want["out"])
    if total:
        check("sum", s, want["sum"])
    check("grad_x", gx, want["grad_x"])
    check("grad_weight", gw, want["grad_weight"])
    check("grad_bias", gb, want["grad_bias"])


# each way of holding a row, its first and last length, and lengths that no vector divides
SIZES = [(1, 1), (3, 4), (5, 7), (2, 8), (2, 17), (37, 32), (9, 33), (70, 40), (64, 96), (11, 128), (13, 129),
         (7, 160), (33, 255), (600, 256), (19, 264), (5, 512), (4, 520), (3, 1024), (3, 1001),
         (2, 2049), (2, 4096), (3, 4104), (5, 6247), (4, 8191), (3, 8192), (2, 8193), (5, 8196), (3, 11247), (3, 11249), (3, 13312), (3, 13316), (3, 14063), (3, 14065), (3, 12001), (2, 16383), (2, 16384), (1, 16392), (2, 32776),
         (1, 70001)]


@pytest.mark.parametrize("dt,pdt", TYPES, ids=IDS)
@pytest.mark.parametrize("N,C", SIZES)
def test_sizes(N, C, dt, pdt):
    for residual, total in ((False, False), (True, True)):
        compare(*operands(N, C, dt, pdt, residual), total)


@pytest.mark.parametrize("dt,pdt", TYPES, ids=IDS)
@pytest.mark.parametrize("N,C", [(44446, 256), (5000, 24), (20011, 77), (3001, 777), (2500, 1024), (1500, 4096)])
def test_many_rows(N, C, dt, pdt):
    compare(*operands(N, C, dt, pdt, residual=True), total=False)


@pytest.mark.parametrize("dt,pdt", TYPES, ids=IDS)
@pytest.mark.parametrize("C", [8, 64, 256, 512, 4096, 8192])
def test_rows_off_a_16_byte_boundary(C, dt, pdt):
    compare(*operands(37, C, dt, pdt, residual=True, offset=1), total=True)


@pytest.mark.parametrize("C", [1, 3, 25, 64, 777])
def test_tensors_off_16_byte_boundaries_by_different_amounts(C):
    """Every tensor starts at its own place in a 16-byte granule, the output too."""
    for dt, pdt in ((BF16, F32), (F32, F32)):
        x, w, b, r, dy, ds = operands(50, C, dt, pdt)
        want = reference(x, w, b, r, 1e-5, dy, ds)

        def moved(t, by):
            flat = torch.full((t.numel() + 16,), 9.0, dtype=t.dtype, device="cuda")
            flat[by:by + t.numel()] = t.flatten()
            return flat, flat[by:by + t.numel()].view(t.shape)

        (_, x), (_, r), (_, dy), (_, ds), (_, w) = (moved(t, by) for t, by in zip((x, r, dy, ds, w), (1, 2, 3, 5, 1)))
        flat, out = moved(torch.zeros_like(x), 7)
        _, s, mean, rstd = binding.msda_layer_norm_forward(x, w, b, r, 1e-5, True, out=out)
        check("out", out, want["out"])
        check("sum", s, want["sum"])
        assert (flat[:7] == 9).all() and (flat[7 + out.numel():] == 9).all()
        gx, gw, gb = binding.msda_layer_norm_backward(dy, x, mean, rstd, w, r, ds)
        for name, g in (("grad_x", gx), ("grad_weight", gw), ("grad_bias", gb)):
            check(name, g, want[name])


@pytest.mark.parametrize("dt", [F32, BF16, F16, F64], ids=IDS)
def test_without_parameters_and_with_one_of_them(dt):
    x, w, b, r, dy, ds = operands(50, 256, dt, dt)
    compare(x, None, None, r, dy, ds, True)
    compare(x, w, None, r, dy, ds, False)
    compare(x, None, b, r, dy, ds, False)


def test_any_subset_of_the_gradients():
    x, w, b, r, dy, ds = operands(300, 256, BF16, F32)
    _, _, mean, rstd = binding.msda_layer_norm_forward(x, w, b, r)
    full = binding.msda_layer_norm_backward(dy, x, mean, rstd, w, r)
    for k in range(8):
        want = tuple(bool(k >> i & 1) for i in range(3))
        got = binding.msda_layer_norm_backward(dy, x, mean, rstd, w, r, want=want)
        for g, f, asked in zip(got, full, want):
            assert torch.equal(g, f) if asked else g is None


@pytest.mark.parametrize("N", [0, 1])
def test_few_rows(N):
    x, w, b, r, dy, ds = operands(max(N, 1), 256, BF16, BF16)
    x, r, dy, ds = x[:N], r[:N], dy[:N], ds[:N]
    out, s, gx, gw, gb = run(x, w, b, r, dy, ds, True)
    assert out.shape == gx.shape == (N, 256)
    if N == 0:
        assert not gw.any() and not gb.any()


def test_eps_and_rows_of_equal_entries():
    x, w, b, r, dy, ds = operands(20, 256, F32, F32, residual=False)
    x[3] = 7.0
    x[4] = 0.0
    for eps in (1e-12, 1e-5, 0.1):
        compare(x, w, b, None, dy, ds, False, eps)
    out = binding.layer_norm(x, w, b, eps=0.0)
    assert out[3].isnan().all() and torch.isfinite(out[5:]).all()


@pytest.mark.parametrize("C", [256, 777, 4096])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_stays_alone(C, value):
    x, w, b, r, dy, ds = operands(40, C, BF16, BF16)
    clean = run(x, w, b, r, dy, ds, True)
    x2 = x.clone()
    x2[17, C // 2] = value
    out, s, gx, gw, gb = run(x2, w, b, r, dy, ds, True)
    keep = torch.arange(40, device="cuda") != 17
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(gx[keep], clean[2][keep])
    assert out[17].isnan().all() and gx[17].isnan().all() and gw.isnan().all()
    assert torch.equal(gb, clean[4])


def test_leading_dimensions_and_one_vector():
    x, w, b, r, dy, ds = operands(24, 256, F32, F32)
    flat = run(x, w, b, r, dy, ds, True)
    shape = (2, 3, 4, 256)
    got = run(x.view(shape), w, b, r.view(shape), dy.view(shape), ds.view(shape), True)
    for f, g in zip(flat, got):
        assert torch.equal(f.reshape(g.shape), g)
    one = binding.layer_norm(x[0], w, b, residual=r[0])
    assert torch.equal(one, flat[0][0])


def test_same_bits_again_and_rows_do_not_depend_on_their_batch():
    x, w, b, r, dy, ds = operands(3000, 256, BF16, BF16)
    first = run(x, w, b, r, dy, ds, True)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, run(x, w, b, r, dy, ds, True)))
    part = run(x[100:117], w, b, r[100:117], dy[100:117], ds[100:117], True)
    assert all(torch.equal(p[100:117], q) for p, q in zip(first[:3], part[:3]))


@pytest.mark.parametrize("C", [250, 256])
def test_offsets_past_32_bits(C):
    N = (1 << 31) // C + 1000
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(N, C, dtype=BF16, device="cuda").normal_(generator=gen)
    dy = torch.empty(N, C, dtype=BF16, device="cuda").normal_(generator=gen)
    w = torch.randn(C, device="cuda", generator=gen)
    b = torch.randn(C, device="cuda", generator=gen)
    out, _, mean, rstd = binding.msda_layer_norm_forward(x, w, b)
    gx, gw, gb = binding.msda_layer_norm_backward(dy, x, mean, rstd, w)
    for rows in (slice(0, 500), slice(N // 2, N // 2 + 500), slice(N - 500, N)):
        want = reference(x[rows], w, b, None, 1e-5, dy[rows])
        check("out", out[rows], want["out"])
        check("grad_x", gx[rows], want["grad_x"])
    exact = torch.zeros(C, dtype=F64, device="cuda")
    size = torch.zeros(C, dtype=F64, device="cuda")
    for part in dy.split(1 << 20):
        exact += part.double().sum(0)
        size += part.double().abs().sum(0)
    # a chain of N / (152 blocks * 3 * 8 warps) rows, then the partial sums
    assert ((gb.double() - exact).abs() <= (100 + N // 256) * 2.0 ** -24 * size).all()


# ------------------------------------------------------------------ autograd

def test_gradients_against_differences():
    x, w, b, r, _, _ = operands(5, 12, F64, F64)
    leaves = [t.requires_grad_() for t in (x, r, w, b)]
    f = lambda x, r, w, b: binding.layer_norm(x, w, b, residual=r, return_sum=True)  # noqa: E731
    assert torch.autograd.gradcheck(f, leaves)
    assert torch.autograd.gradcheck(lambda x: binding.layer_norm(x), [x])


@pytest.mark.parametrize("dt,pdt", TYPES, ids=IDS)
def test_autograd(dt, pdt):
    x, w, b, r, dy, ds = operands(60, 256, dt, pdt)
    want = reference(x, w, b, r, 1e-5, dy, ds)
    leaves = [t.requires_grad_() for t in (x, r, w, b)]
    out, s = binding.layer_norm(x, w, b, residual=r, return_sum=True)
    gx, gr, gw, gb = torch.autograd.grad([out, s], leaves, [dy, ds])
    assert torch.equal(gx, gr)
    for name, g in (("out", out), ("sum", s), ("grad_x", gx), ("grad_weight", gw), ("grad_bias", gb)):
        check(name, g, want[name])


def test_autograd_uses_of_one_output():
    x, w, b, r, dy, ds = operands(60, 256, F32, F32)
    leaves = [t.requires_grad_() for t in (x, r, w, b)]
    out, s = binding.layer_norm(x, w, b, residual=r, return_sum=True)
    got = torch.autograd.grad(s, leaves, ds, allow_unused=True, retain_graph=True)
    assert torch.equal(got[0], ds) and got[2] is None and got[3] is None
    got = torch.autograd.grad(out, leaves, dy)
    check("grad_x", got[0], reference(x, w, b, r, 1e-5, dy)["grad_x"])


def test_autograd_takes_strides_broadcast_gradients_and_frozen_parameters():
    x, w, b, r, dy, ds = operands(64, 64, F32, F32)
    xt = x.t().contiguous().t().requires_grad_()
    out = binding.layer_norm(xt, w, b, residual=r)
    assert torch.equal(out, binding.layer_norm(x, w, b, residual=r))
    g, = torch.autograd.grad(out.sum(), [xt])
    check("grad_x", g, reference(x, w, b, r, 1e-5, torch.ones_like(x))["grad_x"])
    w.requires_grad_()
    gw, = torch.autograd.grad(binding.layer_norm(x, w, b, residual=r), [w], dy)
    check("grad_weight", gw, reference(x, w, b, r, 1e-5, dy)["grad_weight"])


def test_the_same_tensor_as_both_summands():
    x, w, b, r, dy, ds = operands(60, 256, F32, F32)
    x.requires_grad_()
    out, s = binding.layer_norm(x, w, b, residual=x, return_sum=True)
    g, = torch.autograd.grad([out, s], [x], [dy, ds])
    want, bound = reference(x, w, b, x, 1e-5, dy, ds)["grad_x"]
    check("grad_x", g, (2 * want, 2 * bound))
    leaf = x.detach().clone().requires_grad_()
    binding.layer_norm(leaf, w, b, residual=leaf).backward(dy)
    want, bound = reference(x, w, b, x, 1e-5, dy)["grad_x"]
    check("grad_x", leaf.grad, (2 * want, 2 * bound))


def test_two_backward_passes_through_one_graph():
    """The second gradients are tensors of their own."""
    x, w, b, r, dy, ds = operands(60, 256, F32, F32)
    leaves = [t.requires_grad_() for t in (x, r, w, b)]
    out = binding.layer_norm(x, w, b, residual=r)
    first = torch.autograd.grad(out, leaves, dy, retain_graph=True)
    kept = [g.clone() for g in first]
    second = torch.autograd.grad(out, leaves, 2 * dy)
    for f, k, s in zip(first, kept, second):
        assert torch.equal(f, k) and torch.equal(s, 2 * k) and f.data_ptr() != s.data_ptr()


def test_second_derivatives_are_refused():
    x, w, b, r, dy, ds = operands(4, 8, F64, F64)
    x.requires_grad_()
    g, = torch.autograd.grad(binding.layer_norm(x, w, b), [x], dy, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


# ------------------------------------------------------- streams and graphs

def test_another_stream_and_captured_graphs():
    a = operands(600, 256, BF16, F32)
    c = operands(900, 777, BF16, F32, seed=1)
    want = [[t.clone() for t in run(*o, True)] for o in (a, c)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, total, mean, rstd = binding.msda_layer_norm_forward(a[0], a[1], a[2], a[3], 1e-5, True, stream=s)
    grads = binding.msda_layer_norm_backward(a[4], a[0], mean, rstd, a[1], a[3], a[5], stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((out, total, *grads), want[0]))
    graphs, outs = [], []
    for o in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*o, True))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):                    # both graphs at once, each with its own workspace
        for t in [t for o in outs for t in o]:
            t.fill_(3.0)
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, w))


@pytest.mark.parametrize("C", [256, 777])
def test_graphed_forward_and_backward(C):
    """Forward and backward captured as two graphs, as a training loop's callables are."""
    from scale_deformable_attention_msda_gb300.layer import LayerNorm
    x, w, b, r, dy, ds = operands(300, C, F32, F32)
    m = LayerNorm(C).cuda()
    with torch.no_grad():
        m.weight.copy_(w)
        m.bias.copy_(b)
    sample = (torch.randn_like(x, requires_grad=True), torch.randn_like(x, requires_grad=True))
    graphed = torch.cuda.make_graphed_callables(m, sample)
    for k in range(3):
        xs, rs = (x + k).requires_grad_(), r.clone().requires_grad_()
        m.zero_grad(set_to_none=True)
        graphed(xs, rs).backward(dy)
        want = reference(xs, w, b, rs, 1e-5, dy)
        for name, g in (("grad_x", xs.grad), ("grad_x", rs.grad), ("grad_weight", m.weight.grad),
                        ("grad_bias", m.bias.grad)):
            check(name, g, want[name])


@pytest.mark.parametrize("pair", [((600, 256, BF16, F32), (900, 777, F16, F16)),
                                  # one kernel with different amounts of shared memory
                                  ((300, 8192, BF16, BF16), (300, 8192, BF16, BF16, False)),
                                  ((300, 8191, F16, F16), (300, 8191, F16, F16, False))])
def test_two_threads_at_once(pair):
    import threading
    sets = [operands(*p, seed=i) for i, p in enumerate(pair)]
    want = [run(*o, o[3] is not None) for o in sets]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(100):
                    got[i] = run(*sets[i], sets[i][3] is not None)
            st.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w) if q is not None)


# ------------------------------------------------------------------- refusals

def test_refusals():
    x, w, b, r, dy, ds = operands(6, 8, F32, F32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layer_norm(x.cpu())
    with pytest.raises(ValueError, match="shape"):
        binding.layer_norm(x, w[:4], b)
    with pytest.raises(ValueError, match="shape"):
        binding.layer_norm(x, w, b, residual=r[:1])            # no broadcasting
    with pytest.raises(ValueError, match="expected"):
        binding.layer_norm(x, w, b, residual=r.half())
    with pytest.raises(ValueError, match="parameters"):
        binding.layer_norm(x, w.half(), b.half())
    with pytest.raises(ValueError, match="expected"):
        binding.layer_norm(x, w, b.double())
    with pytest.raises(ValueError, match="on cpu"):
        binding.layer_norm(x, w.cpu(), b)
    with pytest.raises(ValueError, match="unsupported dtype"):
        binding.layer_norm(x.int())
    with pytest.raises(ValueError, match="return_sum"):
        binding.layer_norm(x, w, b, return_sum=True)
    with pytest.raises(ValueError, match="channel"):
        binding.layer_norm(x[0, 0])
    with pytest.raises(ValueError, match="contiguous"):
        binding.msda_layer_norm_forward(x.t())
    with pytest.raises(ValueError, match="overlaps"):
        binding.msda_layer_norm_forward(x, w, b, out=x)
    for eps in (-1.0, float("nan")):
        with pytest.raises(binding.MSDAError, match="SHAPE"):
            binding.layer_norm(x, w, b, eps=eps)
    with pytest.raises(binding.MSDAError, match="SHAPE"):
        binding.layer_norm(x[:, :0])
    _, _, mean, rstd = binding.msda_layer_norm_forward(x, w, b)
    with pytest.raises(ValueError, match="mean"):
        binding.msda_layer_norm_backward(dy, x, mean[:3], rstd, w)
    with pytest.raises(ValueError, match="expected"):
        binding.msda_layer_norm_backward(dy, x, mean.double(), rstd, w)


# --------------------------------------------------------- range-checked build

@pytest.mark.parametrize("N,C", [(1, 1), (5, 7), (70, 40), (600, 256), (44446, 256), (9, 777), (1001, 33),
                                 (19, 4104), (7, 8191), (3, 12001), (3, 13312), (2, 16384), (3, 32776)])
def test_accesses_stay_in_bounds(N, C):
    binding.use_library(build.CHECKED_LIBRARY)
    try:
        for dt, pdt in ((F32, F32), (BF16, F32), (F64, F64)):
            compare(*operands(N, C, dt, pdt, residual=True), total=True)
            compare(*operands(N, C, dt, pdt, residual=False, offset=1), total=False)
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()
