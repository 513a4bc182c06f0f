"""Layer norm in float64 with, beside each output, how far a result computed in
fp32 (or fp64) and rounded once may be from it: first-order bounds of the
rounding errors, elementwise.

u is half a step of the arithmetic's type, h half a step of the stored type.
A sum of terms t_i added in chains and trees of at most D additions is off by
at most D*u*sum|t_i|.
"""
import torch

HALF = {torch.float64: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8,
        torch.float16: 2.0 ** -11}
# half the distance between the smallest numbers of a type, the error of a rounding near zero
TINY = {torch.float64: 2.0 ** -1075, torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134,
        torch.float16: 2.0 ** -25}
SECOND = 1.05      # second-order terms


def rounded(value, error, dtype):
    """Bound after one rounding to `dtype` of something `error` away from `value`."""
    return SECOND * (error + HALF[dtype] * (value.abs() + error)) + TINY[dtype]


def reference(x, weight, bias, residual=None, eps=1e-5, grad_out=None, grad_sum=None):
    """{name: (value, bound)} for out, sum and, with grad_out, the three gradients."""
    dt = x.dtype
    pdt = weight.dtype if weight is not None else bias.dtype if bias is not None else dt
    C = x.shape[-1]
    x, r = x.detach().double().reshape(-1, C), None if residual is None else residual.detach().double().reshape(-1, C)
    N = x.shape[0]
    w = torch.ones(C, dtype=torch.float64, device=x.device) if weight is None else weight.detach().double()
    b = torch.zeros_like(w) if bias is None else bias.detach().double()
    u = HALF[torch.float64 if dt == torch.float64 else torch.float32]
    D = 64 + C // 256            # additions on the way of one term of a row's sum, at most
    s = x if r is None else x + r
    biggest = (x.abs() + (0 if r is None else r.abs())).amax(-1, keepdim=True)
    mean = s.mean(-1, keepdim=True)
    rstd = ((s - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (s - mean) * rstd
    # s and the mean are off by (D + 2) u biggest together, and so is a distance from the mean;
    # 1/rstd is the root of a mean of squares of those distances
    far = (D + 2) * u * biggest * rstd
    rel_r = far + (D + 7) * u
    e_xh = far + xh.abs() * (rel_r + u)
    y = xh * w + b
    got = {"out": (y, rounded(y, w.abs() * e_xh + 2 * u * ((xh * w).abs() + b.abs()), dt)),
           "sum": (s, rounded(s, u * s.abs(), dt))}
    if grad_out is None:
        return got
    dy = grad_out.detach().double().reshape(-1, C)
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    e_c1 = (D + 2) * u * g.abs().mean(-1, keepdim=True)
    e_c2 = (D + 3) * u * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * e_xh).mean(-1, keepdim=True)
    inner = g - c1 - xh * c2
    dx = rstd * inner
    e_dx = rstd * (4 * u * (g.abs() + c1.abs() + (xh * c2).abs()) + e_c1 + xh.abs() * e_c2 + c2.abs() * e_xh)
    e_dx = e_dx + rel_r * dx.abs()
    if grad_sum is not None:
        dx = dx + grad_sum.detach().double().reshape(-1, C)
        e_dx = e_dx + 2 * u * dx.abs()
    rows = 100 + N // 256        # additions on the way of one term of a column's sum
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (dy.abs() * e_xh).sum(0) + rows * u * (dy * xh).abs().sum(0)
    e_db = rows * u * dy.abs().sum(0)
    got["grad_x"] = (dx, rounded(dx, e_dx, dt))
    got["grad_weight"] = (dw, rounded(dw, e_dw, pdt))
    got["grad_bias"] = (db, rounded(db, e_db, pdt))
    return got


def check(name, got, expected):
    value, bound = expected
    got = got.detach().double().reshape(value.shape)
    off = (got - value).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values out of bounds, worst "
                           f"{float((off / bound).max()):.3g} times the bound")
