"""Attention and its gradients in float64 with, beside each output, how far a result
computed in fp32 with 16-bit weights may be from it: first-order bounds of the
rounding errors, elementwise.

u is half a step of fp32, h half a step of the data's type (of a weight that is
rounded to it as an operand; 0 for fp32 data). A sum of terms t_i added in chains
of at most n additions is off by at most n u sum|t_i|; the tensor cores may cut
instead of round, which counts as 2u.
"""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
U = 2.0 ** -24
SECOND = 1.1       # second-order terms


def rounded(value, error, dtype):
    """Bound after one rounding to `dtype` of something `error` away from `value`."""
    return SECOND * (error + HALF[dtype] * (value.abs() + error)) + TINY[dtype]


def reference(q, k, v, mask=None, scale=None, grad_out=None, exact_out=False):
    """{name: (value, bound)} of out, lse and, with grad_out, gq, gk, gv. exact_out: the
    backward is given the exact out (in two parts for 16-bit data) and lse rounded to fp32;
    else those that a forward computed."""
    dt = q.dtype
    h = 0.0 if dt == torch.float32 else HALF[dt]
    B, Q, M, D = q.shape
    S, N = k.shape[1:3]
    g = M // N
    scale = D ** -0.5 if scale is None else scale
    qd, kd, vd = (t.detach().double().transpose(1, 2) for t in (q, k, v))
    kd, vd = kd.repeat_interleave(g, 1), vd.repeat_interleave(g, 1)
    on = torch.ones(B, M, Q, S, dtype=torch.bool, device=q.device) if mask is None else mask.expand(B, M, Q, S)
    # what lies in masked places has no part
    s = torch.where(on, scale * (qd.nan_to_num() @ kd.nan_to_num().mT), -math.inf)
    some = on.any(-1, keepdim=True)
    lse = torch.where(some, torch.logsumexp(torch.where(some, s, 0.0), -1, keepdim=True), -math.inf)
    p = torch.where(on, torch.exp(s - torch.where(some, lse, 0.0)), 0.0)
    vz = vd.nan_to_num(0.0, 0.0, 0.0)
    out = p @ vz
    # a score, in the exponent: products in chains of D + 4, then times scale
    size = scale * (qd.nan_to_num(0.0, 0.0, 0.0).abs() @ kd.nan_to_num(0.0, 0.0, 0.0).abs().mT)
    es = ((D + 8) * 2 * U * torch.where(on, size, 0.0)).amax(-1, keepdim=True) if S else torch.zeros_like(lse)
    chain = 64 + S / 32            # additions on the way of one term of a row's sums
    ep = 2 * es + 2.0 ** -21 + chain * U + 4 * U * torch.where(some, s.masked_fill(~on, 0).abs().amax(-1, keepdim=True) if S else lse, 0.0)
    e_out = (p * (h + ep + chain * 2 * U)) @ vz.abs()
    if dt == torch.float16:        # weights below fp16's smallest
        e_out = e_out + 2.0 ** -31 * vz.abs().sum(-2, keepdim=True)
    flat = lambda t: t.transpose(1, 2).reshape(B, Q, M * D)      # noqa: E731
    result = {"out": (flat(out), rounded(flat(out), flat(e_out), dt)),
              "lse": (lse[..., 0], SECOND * (es + ep + 2 * U * lse.abs().nan_to_num(0, 0, 0))[..., 0] + 1e-30)}
    if grad_out is None:
        return result
    go = grad_out.detach().double().view(B, Q, M, D).transpose(1, 2)
    gz = torch.where(some, go, 0.0)          # a query without keys has no part
    dp = gz @ vz.mT
    delta = (gz * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    two = (D + 8) * 2 * U
    e_dp = two * (gz.abs() @ vz.abs().mT)
    e_delta = two * (gz.abs() * out.abs()).sum(-1, keepdim=True) + 4 * U * delta.abs()
    known = HALF[dt] ** 2 if dt != torch.float32 else U
    e_delta = e_delta + (gz.abs() * (known * out.abs() + TINY[dt] + (0 if exact_out else e_out))).sum(-1, keepdim=True)
    ebp = ep + 4 * U * torch.where(some, lse.abs(), 0.0)         # with lse as an fp32 number
    e_p = p * (h + ebp)
    e_ds = ds.abs() * (h + ebp) + p * (e_dp + e_delta)
    if dt == torch.float16:
        largest = gz.norm(dim=-1).amax() * vz.norm(dim=-1).amax() if gz.numel() and vz.numel() else 0.0
        e_p, e_ds = e_p + 2.0 ** -38 * on, e_ds + 2.0 ** -36 * largest * on
    qz, kz = qd.nan_to_num(0.0, 0.0, 0.0), kd.nan_to_num(0.0, 0.0, 0.0)
    long = lambda n: (64 + n / 8) * 2 * U                        # noqa: E731
    gq, e_gq = scale * (ds @ kz), scale * ((e_ds + long(S) * ds.abs()) @ kz.abs())
    over = lambda t: t.view(B, N, g, S, D).sum(2)                # noqa: E731
    gv, e_gv = over(p.mT @ gz), over((e_p + long(Q * g) * p).mT @ gz.abs())
    gk, e_gk = scale * over(ds.mT @ qz), scale * over((e_ds + long(Q * g) * ds.abs()).mT @ qz.abs())
    back = lambda t: t.transpose(1, 2)                           # noqa: E731
    for name, value, error in (("gq", gq, e_gq), ("gk", gk, e_gk), ("gv", gv, e_gv)):
        result[name] = (back(value), rounded(back(value), back(error), dt))
    return result


def check(name, got, want):
    value, bound = want
    assert got.shape == value.shape, name
    same = got.double() == value             # infinities
    off = torch.where(same, torch.zeros_like(value), (got.double() - value).abs())
    assert torch.isfinite(off).all(), f"{name}: not finite"
    over = off > bound
    if over.any():
        at = tuple(over.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(over.sum())} of {over.numel()} over their bound, first at {at}: "
                             f"{float(got[at])}, not {float(value[at])} within {float(bound[at])}")
