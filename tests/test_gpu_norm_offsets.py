"""Layer norm of rows whose entries lie far from zero beside their spread, and of rows of
equal entries: the mean's own roundings must not show in the outputs.

Bounds, first order. u: half a step of the arithmetic; D: additions on the way of one term
of a row's sum, at most. The first mean is off by at most delta = (D + 2) u max|s|. The
distances from it, each rounded once, have a mean that is found within
e_shift = (D + 3) u (mean|s - mean| + delta), and are corrected by it: a distance is off by
e_shift and two roundings, whatever the mean's size. The mean of the squared distances less
the square of that shift is off by e_var = (D + 4) u (var + delta^2) + 2 delta e_shift.
Rows whose mean is within 2 / rstd of zero may keep the first mean: off by
(D + 2) u max|s| rstd <= 2 (D + 2) u in the normalised row where all entries are equal, and by
delta otherwise; rstd is that of the distances from it, whose squares hold delta^2 more.
The stored mean is rounded once more, u |mean|, which the backward sees.
"""
import pytest
import torch

from norm_reference import HALF, check, rounded
from scale_deformable_attention_msda_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64
IDS = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731
# every way of holding a row, and lengths whose reciprocal is not exact
COLUMNS = [2, 3, 7, 96, 256, 333, 777, 1001, 2560, 4096, 4097, 8192, 12001, 16384, 16392, 32776, 70001]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def parameters(C, pdt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + C)
    return [(shift + 0.3 * torch.randn(C, device="cuda", generator=gen)).to(pdt) for shift in (1.0, 0.0)]


@pytest.mark.parametrize("dt", [F32, BF16, F16, F64], ids=IDS)
@pytest.mark.parametrize("C", COLUMNS)
def test_rows_of_equal_entries(C, dt):
    """Their distances from the mean are zero: the output is the bias, the mean the entry,
    exactly where entries are over 2 / rstd."""
    w, b = parameters(C, dt)
    values = torch.tensor([10000.1, 100.1, 0.1, 3.3, -77.7, 1e-3, 7.0, 0.0], device="cuda", dtype=F64).to(dt)
    x = values[:, None].expand(-1, C).contiguous()
    half = (values.double() / 2).to(dt)[:, None].expand(-1, C).contiguous()
    for eps in (1e-5, 1e-12):
        for args in (dict(x=x), dict(x=half, residual=half)):
            out, _, mean, _ = binding.msda_layer_norm_forward(weight=w, bias=b, eps=eps, **args)
            s = args["x"].double() + (args["residual"].double() if "residual" in args else 0)
            far = s[:, 0].abs() * eps ** -0.5 > 2.1
            assert torch.equal(mean.double()[far], s[far, 0])
            assert torch.equal(out[far], b.expand_as(out)[far])
            first = (66 + C // 256) * HALF[F64 if dt == F64 else F32]
            check("mean", mean, (s[:, 0], 1.05 * first * s[:, 0].abs()))
            e_out = (2.1 * first * w.double().abs()).expand_as(s)
            check("out", out, (b.double().expand_as(s), rounded(b.double().expand_as(s), e_out, dt)))
    assert binding.layer_norm(x, w, b, eps=0.0).isnan().all()


def reference(x, w, b, eps, dy):
    dt, pdt, C = x.dtype, w.dtype, x.shape[-1]
    s, w, b, dy = x.double(), w.double(), b.double(), dy.double()
    u, D = HALF[F64 if dt == F64 else F32], 64 + C // 256
    mean = s.mean(-1, keepdim=True)
    far = s - mean
    far = far - far.mean(-1, keepdim=True)       # (rounding of the mean itself, for fp64)
    var = far.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = far * rstd
    delta = (D + 2) * u * s.abs().amax(-1, keepdim=True)
    e_shift = (D + 3) * u * (far.abs().mean(-1, keepdim=True) + delta)
    near = s.abs().amax(-1, keepdim=True) * rstd < 2.1      # no correction is owed
    e_shift = torch.where(near, delta, e_shift)
    e_var = (D + 4) * u * (var + delta.square()) + 2 * delta * e_shift
    rel_r = e_var / 2 / (var + eps) + 5 * u
    e_xh = rstd * (e_shift + u * (2 * far.abs() + delta)) + xh.abs() * (rel_r + 2 * u)
    y = xh * w + b
    got = {"out": (y, rounded(y, w.abs() * e_xh + 2 * u * ((xh * w).abs() + b.abs()), dt))}
    # the backward takes its distances from the stored mean
    e_xh = rstd * (e_shift + u * (mean.abs() + e_shift + far.abs())) + xh.abs() * (rel_r + 2 * u)
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    e_c1 = (D + 2) * u * g.abs().mean(-1, keepdim=True)
    e_c2 = (D + 3) * u * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * e_xh).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    e_dx = rstd * (4 * u * (g.abs() + c1.abs() + (xh * c2).abs()) + e_c1 + xh.abs() * e_c2 + c2.abs() * e_xh)
    got["grad_x"] = (dx, rounded(dx, e_dx + rel_r * dx.abs(), dt))
    rows = 100 + x.shape[0] // 256
    dw = (dy * xh).sum(0)
    got["grad_weight"] = (dw, rounded(dw, (dy.abs() * e_xh).sum(0) + rows * u * (dy * xh).abs().sum(0), pdt))
    return got


# offset and step of the entries, exact in the type: the spread is 37 steps
FAR = [(F32, 10000.0, 2.0 ** -6), (F32, -1e6, 2.0 ** -3), (F32, 3.0, 2.0 ** -16), (BF16, 256.0, 2.0),
       (F16, 1024.0, 1.0), (F64, 1e9, 2.0 ** -12)]


@pytest.mark.parametrize("dt,offset,step", FAR, ids=IDS)
@pytest.mark.parametrize("C", COLUMNS)
def test_rows_far_from_zero(C, dt, offset, step):
    gen = torch.Generator(device="cuda").manual_seed(C)
    k = torch.randint(-64, 65, (9, C), device="cuda", generator=gen)
    if dt in (BF16, F16):
        k = k.abs()                              # up from a power of two: exact
    x = (offset + k.double() * step).to(dt)
    assert torch.equal(x.double(), offset + k.double() * step)
    dy = torch.randn(9, C, device="cuda", generator=gen).to(dt)
    w, b = parameters(C, F64 if dt == F64 else F32)
    out, _, mean, rstd = binding.msda_layer_norm_forward(x, w, b)
    grads = binding.msda_layer_norm_backward(dy, x, mean, rstd, w)
    want = reference(x, w, b, 1e-5, dy)
    check("out", out, want["out"])
    check("grad_x", grads[0], want["grad_x"])
    check("grad_weight", grads[1], want["grad_weight"])


@pytest.mark.parametrize("C", [256, 333, 4096, 12001, 32776])
@pytest.mark.parametrize("dt,size", [(F32, 1e20), (BF16, 1e30), (F64, 1e200), (F32, 3e38)], ids=IDS)
def test_rows_that_leave_the_arithmetics_range(C, dt, size):
    """Squares that overflow make their row not finite, and no other."""
    gen = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn(20, C, device="cuda", generator=gen, dtype=F64).to(dt)
    w, b = parameters(C, dt)
    clean = binding.layer_norm(x, w, b)
    x[7] = size
    x[7, ::2] = -size
    out = binding.layer_norm(x, w, b)
    keep = torch.arange(20, device="cuda") != 7
    assert torch.equal(out[keep], clean[keep]) and not out[7].isfinite().any()


@pytest.mark.parametrize("dt", [F32, BF16, F64], ids=IDS)
@pytest.mark.parametrize("C", COLUMNS)
def test_equal_rows_without_eps(C, dt):
    """NaN whatever the entry's size, where squares of the mean or the distances vanish too."""
    values = torch.tensor([0.0, 1e-38, 1e-30, 1.1e-22, 1e-10, -3.3, 1e10, 1.7e19, 3e34], device="cuda", dtype=F64).to(dt)
    x = values[:, None].expand(-1, C).contiguous()
    assert binding.layer_norm(x, eps=0.0).isnan().all()


@pytest.mark.parametrize("dt", [F32, BF16, F64], ids=IDS)
@pytest.mark.parametrize("C", [256, 333, 4096, 12001, 32776])
def test_an_eps_past_the_arithmetics_range(C, dt):
    """rstd is zero then, not NaN: the output is the bias."""
    w, b = parameters(C, dt)
    x = torch.randn(5, C, device="cuda").to(dt) + 3
    for eps in (1e39, float("inf")):
        if eps == 1e39 and dt == F64:
            continue                     # in range: rstd is 3e-20
        assert torch.equal(binding.layer_norm(x, w, b, eps=eps), b.expand_as(x))


# lengths for each number of lanes and warps that hold a row, and of places that each has
LENGTHS = [8, 16, 20, 24, 32, 40, 48, 64, 72, 100, 128, 160, 192, 257, 264, 384, 512, 513, 640, 768, 1000, 1024, 1025,
           1536, 2048, 2504, 4104, 5000, 6000, 8000, 10000, 13312]


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("C", LENGTHS)
def test_far_and_near_rows_side_by_side(C, dt):
    """Rows far from zero, equal rows and ordinary ones in turn: each as if it were alone, to
    the bit, and within the bounds."""
    gen = torch.Generator(device="cuda").manual_seed(C)
    N = 203
    k = torch.randint(0, 65, (N, C), device="cuda", generator=gen).double()
    offset, step = {F32: (10000.0, 2.0 ** -6), BF16: (256.0, 2.0), F16: (1024.0, 1.0)}[dt]
    x = torch.randn(N, C, device="cuda", generator=gen).to(dt)
    x[1::3] = (offset + k[1::3] * step).to(dt)
    x[2::7] = 300.0
    w, b = parameters(C, F32)
    out, _, mean, rstd = binding.msda_layer_norm_forward(x, w, b)
    check("out", out, reference(x, w, b, 1e-5, torch.zeros_like(x))["out"])
    for i in range(0, 21):
        one = binding.msda_layer_norm_forward(x[i:i + 1], w, b)
        if x[i:i + 1].data_ptr() % 16 == 0 or C * dt.itemsize % 16:      # the same form of the kernels
            assert torch.equal(one[0][0], out[i]) and torch.equal(one[2][0], mean[i]) and torch.equal(one[3][0], rstd[i])
