"""Clipping where the factor itself leaves fp32's normal numbers. Bounds as in
test_gpu_gradnorm.py: 33 u of the norm, two roundings of the factor, the product's."""
import math

import pytest
import torch

from norm_reference import HALF, TINY
from scale_deformable_attention_msda_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dt,out", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=str)
@pytest.mark.parametrize("max_norm", [1e-1, 1e-3, 1e-6, 1e-12, 1e-20])
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("more", [[], [1_500_001]], ids=["one launch", "two"])
def test_a_factor_below_the_normal_numbers(dt, out, max_norm, kind, more):
    """Entries near fp32's largest, a norm that a product with a subnormal factor would
    take digits from (1e-3 of 1e38 is 1e-41, of 2^-149 steps 1e-4 of it)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    grads = [(torch.randn(n, device="cuda", generator=gen, dtype=F64) * 1e34).to(dt) for n in [9, 4097, 31] + more]
    grads[0][3] = 2e37
    flat = torch.cat([g.double() for g in grads])
    norm = float(flat.abs().max() if kind == math.inf else flat.square().sum().sqrt())
    outs = [torch.empty(g.shape, device="cuda", dtype=out) for g in grads]
    got = binding.msda_clip_grad_norm(binding.GradientBuffers(grads, out=outs), max_norm, kind)
    u = 2.0 ** -24
    assert abs(float(got) - norm) <= 34 * u * norm
    for g, o in zip(grads, outs):
        want = g.double() * (max_norm / (norm + 1e-6))
        tol = (36 * u + HALF[out]) * 1.01 * want.abs() + TINY[out]
        assert ((o.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("max_norm", [1e-10, 1e-100])
def test_fp64(max_norm):
    """The largest entry of 1e300 gives a factor below fp64's normal numbers."""
    g = torch.tensor([1e300, -3e299, 7e250, 1.0], device="cuda", dtype=F64)
    out = torch.empty_like(g)
    norm = binding.msda_clip_grad_norm(binding.GradientBuffers([g], out=[out]), max_norm, math.inf)
    assert float(norm) == 1e300
    want = (g / 1e300) * max_norm        # two roundings in fp64, as the kernel's quotient and product
    assert ((out - want).abs() <= 6 * 2.0 ** -53 * want.abs() + TINY[F64]).all()


def test_factors_that_are_ordinary_change_no_bit():
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.randn(100_003, device="cuda", generator=gen)
    out = torch.empty_like(g)
    norm = float(binding.msda_clip_grad_norm(binding.GradientBuffers([g], out=[out]), 0.5))
    near = torch.tensor([0.5 / (norm + 1e-6)], dtype=F64).float()
    # the factor from the norm's fp64 value, which the returned float is a rounding of
    steps = [near, torch.nextafter(near, near * 0), torch.nextafter(near, near * 2)]
    assert any(torch.equal(out, g * f.cuda()) for f in steps)


def clipped(value, max_norm, kind=2.0, dt=F64):
    g = torch.tensor([value], device="cuda", dtype=dt)
    binding.msda_clip_grad_norm([g], max_norm, kind)
    return g


def test_a_norm_just_under_the_limit():
    """The factor is max_norm / (norm + 1e-6): within 1e-6 of the limit it is below one."""
    for dt in (F32, F64):
        for value, max_norm in ((1.0 - 2e-6, 1.0), (0.5, 0.5 + 2e-6), (0.0, 1e-7), (3.0, math.inf)):
            assert torch.equal(clipped(value, max_norm, dt=dt), torch.tensor([value], device="cuda", dtype=dt))
        for value, max_norm in ((1.0 - 5e-7, 1.0), (0.5, 0.5), (5e-8, 1e-7)):
            held = torch.tensor([value], dtype=dt).double()
            want = held * (max_norm / (held + 1e-6))
            got = clipped(value, max_norm, dt=dt).double().cpu()
            assert got < held
            # one entry: its square and the root in fp64 or fp32, the factor, the product
            assert (got - want).abs() <= 6 * HALF[dt] * want


def test_what_the_header_says_of_infinities():
    assert clipped(math.inf, math.inf).isnan() and clipped(math.inf, 1.0).isnan()
    g = torch.tensor([math.inf, 2.0], device="cuda")
    binding.msda_clip_grad_norm([g], 1.0)
    assert g[0].isnan() and g[1] == 0
    # the float is past its range, the norm that makes the factor is not
    g = torch.full((100,), 3e38, device="cuda")
    assert binding.msda_clip_grad_norm([g], 1.0) == math.inf
    assert ((g.double() - 0.1).abs() <= 40 * 2.0 ** -24 * 0.1).all()
    assert binding.msda_grad_norm([torch.full((2,), 1e160, device="cuda", dtype=F64)]) == math.inf


def test_a_double_norm_of_fp32_entries():
    """Its fp32 share is within the bound of fp32 lists."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    g = torch.randn(1_000_003, device="cuda", generator=gen)
    d = torch.full((1,), 1e-3, device="cuda", dtype=F64)
    norm = binding.msda_grad_norm([g, d])
    want = (g.double().square().sum() + 1e-6).sqrt()
    assert norm.dtype == F64 and abs(norm - want) <= (33 * 2.0 ** -24) * want
