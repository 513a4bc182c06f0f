"""Layer norm's backward where a thread's places hold no data: lengths that leave lanes
idle, and row counts that leave groups without a row. What such a place computes must not
reach a result, however large mean * rstd is."""
import pytest
import torch

from norm_reference import check
from scale_deformable_attention_msda_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "off"])
@pytest.mark.parametrize("C", [2, 7, 24, 40, 72, 200, 333, 640, 777, 1000, 1001, 2504, 5000, 8000, 8191, 12000])
def test_huge_equal_rows(C, offset, dt):
    """Rows of equal entries near 2e36 with eps 1e-5 (1e33 with 1e-12): mean * rstd leaves
    fp32's range, the true distances are zero, so xh is zero, grad_x is
    rstd * (g - mean(g)) and grad_weight gets nothing from them."""
    for eps, size in ((1e-5, 2e36), (1e-12, 1e33)):
        for N in (1, 5, 700):
            gen = torch.Generator(device="cuda").manual_seed(N * C)
            flat = torch.full((N * C + offset,), size, device="cuda", dtype=dt)
            x = flat[offset:].view(N, C)
            # grad_out so small that rstd times it stays in range; fp32 sums of up to 12,000
            dy = (torch.randn(N * C + offset, device="cuda", generator=gen) * 1e-3).to(dt)[offset:].view(N, C)
            w = torch.randn(C, device="cuda", generator=gen)
            _, _, mean, rstd = binding.msda_layer_norm_forward(x, w, None, eps=eps)
            # the statistics as they are: this is about the backward alone
            mean.copy_(x[:, 0].float())
            rstd.fill_(eps ** -0.5)
            gx, gw, gb = binding.msda_layer_norm_backward(dy, x, mean, rstd, w)
            g, r = dy.double() * w.double(), float(rstd[0].double())
            want = r * (g - g.mean(-1, keepdim=True))
            # a product, a sum of at most 64 + C/256 additions, two operations after
            u, half = 2.0 ** -24, 2.0 ** -24 if dt == torch.float32 else 2.0 ** -8
            bound = r * u * ((70 + C // 256) * g.abs().mean(-1, keepdim=True) + 4 * (g.abs() + g.mean(-1, keepdim=True).abs()))
            check("grad_x", gx, (want, 1.05 * (bound + half * (want.abs() + bound))))
            assert not gw.any()
            db = dy.double().sum(0)
            # bias gradients are fp32: sums of N terms in at most 100 + N/256 additions
            check("grad_bias", gb, (db, 1.05 * (101 + N // 256) * u * dy.double().abs().sum(0)))
