"""Masked attention of operands that are not finite, in allowed and in masked places: what it
gives, and that it takes no more than a small multiple of an ordinary call."""
import pytest
import torch

from attention_reference import check, reference
from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, IDS, _lib, operands  # noqa: F401

pytestmark = pytest.mark.gpu


def seconds(call):
    call()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = float("inf")
    for _ in range(3):
        torch.cuda.synchronize()
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) * 1e-3)
    return best


def padded(B, S, ends):
    return (torch.arange(S, device="cuda") < torch.tensor(ends, device="cuda")[:, None])[:, None, None, :]


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("sizes", [(2, 1024, 1000, 8, 4, 32), (2, 700, 1024, 4, 1, 128)], ids=str)
def test_time(sizes, dt):
    """Overflowed gradients and activations in allowed places, as loss scaling meets them, cost a
    pass over the columns at the most; what lies in masked places, one computation of each row that
    it meets: ten and three hundred times an ordinary call, and no more."""
    B, Q, S, M, N, D = sizes
    q, k, v, go, _ = operands(*sizes, dt, seed=1)
    mask = padded(B, S, [S, S - 100])

    def times(q, k, v, go):
        out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
        return (seconds(lambda: binding.msda_attention_forward(q, k, v, mask=mask, rest=True)),
                seconds(lambda: binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, rest=rest)))
    plain = times(q, k, v, go)
    bad_go, bad_v, bad_q = go.clone(), v.clone(), q.clone()
    bad_go[:, ::50] = float("inf")
    bad_v[:, 5] = float("nan")
    bad_q[0, 3] = float("nan")
    everywhere = [torch.full_like(t, float("nan")) for t in (q, k, v, go)]
    for operand in ((q, k, v, bad_go), (q, k, bad_v, go), (bad_q, k, v, go), everywhere):
        for took, ordinary in zip(times(*operand), plain):
            assert took <= 10 * ordinary + 1e-4
    behind = [t.clone() for t in (k, v)]
    for t in behind:
        t[1, S - 100:] = float("nan")
    for took, ordinary in zip(times(q, *behind, go), plain):
        assert took <= 300 * ordinary


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("sizes", [(2, 150, 300, 4, 2, 32), (1, 260, 140, 2, 1, 128), (2, 1, 900, 4, 1, 64), (2, 70, 90, 3, 3, 64)], ids=str)
def test_allowed_and_masked_places(sizes, bad, dt):
    """Bad values in masked places beside bad values in allowed ones: rows whose allowed pairs are
    all finite are as if there were none, and the others are not finite."""
    if bad == 3e38 and dt == F16:
        pytest.skip("fp16 has no such number")
    B, Q, S, M, N, D = sizes
    q, k, v, go, gen = operands(*sizes, dt, seed=2)
    mask = torch.rand(B, M, Q, S, device="cuda", generator=gen) < 0.7
    mask[..., S // 2:S // 2 + 4] = False             # keys that no query attends: may hold anything
    mask[..., 9] = False
    mask[:, :, Q // 3, 9] = True                     # a key that one query of each head attends
    if Q > 20:
        mask[:, :, 7] = False                        # a query without keys
    clean = reference(q, k, v, mask, None, go)
    dk, dv, dq, dgo = k.clone(), v.clone(), q.clone(), go.clone()
    dk[:, S // 2:S // 2 + 4] = bad
    dv[:, S // 2:S // 2 + 4] = bad
    if Q > 20:
        dq[:, 7], dgo[:, 7] = bad, bad
    kept = torch.ones(Q, dtype=torch.bool, device="cuda")
    out, lse, rest = binding.msda_attention_forward(dq, dk, dv, mask=mask, rest=True)
    check("out", out, clean["out"])
    check("lse", lse, clean["lse"])
    for name, got in zip(("gq", "gk", "gv"), binding.msda_attention_backward(dgo, dq, dk, dv, out, lse, mask=mask, rest=rest)):
        check(name, got, clean[name])
    if bad == 3e38:
        return
    dv[:, 9] = bad                                   # now also in an allowed place
    kept[Q // 3] = False
    out, lse, rest = binding.msda_attention_forward(dq, dk, dv, mask=mask, rest=True)
    value, bound = clean["out"]
    check("out", out[:, kept], (value[:, kept], bound[:, kept]))
    assert not torch.isfinite(out[:, ~kept]).any()
    grads = binding.msda_attention_backward(dgo, dq, dk, dv, out, lse, mask=mask, rest=rest)
    value, bound = clean["gq"]
    check("gq", grads[0][:, kept], (value[:, kept], bound[:, kept]))
    assert not torch.isfinite(grads[0][:, ~kept]).any()


@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=IDS)
def test_the_same_without_and_with_a_mask(dt):
    """Where a mask allows all that is there, what is not finite is where it is without a mask."""
    q, k, v, go, _ = operands(2, 200, 260, 4, 2, 64, dt, seed=3)
    go.view(2, 200, 4, 64)[0, 17, 1, 3] = float("inf")
    v[1, 30, 0, 5] = float("inf")
    q[1, 99, 2, 7] = float("nan")
    mask = torch.ones(2, 1, 200, 260, dtype=torch.bool, device="cuda")
    mask[:, :, 150] = False
    mask[:, :, :, 250:] = False
    plain = [q[:, :], k[:, :250], v[:, :250]]
    out, lse, rest = binding.msda_attention_forward(*plain, rest=True)
    masked, lse2, rest2 = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
    at = torch.arange(200, device="cuda") != 150
    assert torch.equal(torch.isfinite(out[:, at]), torch.isfinite(masked[:, at]))
    assert torch.equal(torch.isfinite(lse[..., at]), torch.isfinite(lse2[..., at]))
    grads = binding.msda_attention_backward(go, *plain, out, lse, rest=rest)
    others = binding.msda_attention_backward(go, q, k, v, masked, lse2, mask=mask, rest=rest2)
    assert torch.equal(torch.isfinite(grads[0][:, at]), torch.isfinite(others[0][:, at]))
    assert (others[0][:, 150] == 0).all()
    for a, b in zip(grads[1:], others[1:]):
        assert torch.equal(torch.isfinite(a), torch.isfinite(b[:, :250]))
        assert (b[:, 250:] == 0).all()
