"""The global gradient norm and clipping against float64.

Bounds. u32 = 2^-24, u64 = 2^-53, h half a step of the stored type. Norm: a lane
adds up to 66 squares in fp32, each product and sum rounded once with fma, so
its sum is off by at most 66 u32 relative; the sums of those are in fp64, or in
pairs of fp32 whose errors (n u32^2) do not show; the square root halves the
relative error, and one rounding to fp32 is added: 33 u32 + u32. fp64: n u64 at most for n entries. Largest entry: exact. Clipped entry: the
norm's error, the factor rounded to fp32, the product and one rounding to the
stored type: 33 u32 + 2 u32 + h relative, and half the smallest number of a type.
"""
import math

import pytest
import torch

from norm_reference import HALF, TINY
from scale_deformable_attention_msda_gb300 import binding, build

pytestmark = pytest.mark.gpu

F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64
U32 = 2.0 ** -24
IDS = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def grads_of(sizes, dt, seed=0, offset=0, scale=0.01):
    """Tensors of the given entry counts, `offset` entries past a 16-byte boundary."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n in sizes:
        t = torch.randn(n + offset, device="cuda", generator=gen, dtype=torch.float64) * scale
        out.append(t.to(dt)[offset:])
    return out


def exact_norm(grads, kind):
    if not sum(g.numel() for g in grads):
        return 0.0
    if kind == math.inf:
        top = torch.stack([g.double().abs().max() for g in grads if g.numel()])
        return float("nan") if top.isnan().any() else float(top.max())
    return float(torch.stack([g.double().square().sum() for g in grads]).sum().sqrt())


def check_norm(norm, grads, kind):
    want, got = exact_norm(grads, kind), float(norm)
    wide = any(g.dtype == F64 for g in grads)
    assert norm.dtype == (F64 if wide else F32) and norm.dim() == 0
    narrow = any(g.dtype != F64 for g in grads)
    n = sum(g.numel() for g in grads)
    tol = (33 * U32 if narrow else 0.0) + (n * 2.0 ** -53 if wide else U32)
    if kind == math.inf:
        tol = 0.0
    assert abs(got - want) <= tol * want, (got, want)
    return want


def check_clipped(before, after, max_norm, norm):
    factor = min(1.0, max_norm / (norm + 1e-6))
    for b, a in zip(before, after):
        want = b.double() * factor
        u = U32 if b.dtype != F64 or any(t.dtype != F64 for t in before) else 2.0 ** -53 * 1e6
        tol = (35 * u + HALF[a.dtype]) * 1.01 * want.abs() + TINY[a.dtype]
        assert ((a.double() - want).abs() <= tol).all()


# one entry, around a vector, a lane row, a unit of 4 KB, many units; empty ones among them
SIZES = [[1], [0, 1, 0], [7, 8, 9], [262144], [262145], [131072], [131073, 0, 4], [511, 512, 513], [1023, 1024, 1025, 2047, 2048, 2049, 4097], [100003],
         [3, 0, 70000, 5, 1, 1, 33, 256, 65536], [1] * 70, [17] * 1500, [2_000_003, 19]]


@pytest.mark.parametrize("dt", [F32, BF16, F16, F64], ids=IDS)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_norm_and_clip_in_place(sizes, dt, kind):
    grads = grads_of(sizes, dt)
    check_norm(binding.msda_grad_norm(grads, kind), grads, kind)
    for max_norm in (0.01, 1e9, 0.0):
        work = [g.clone() for g in grads]
        norm = binding.msda_clip_grad_norm(work, max_norm, kind)
        want = check_norm(norm, grads, kind)
        check_clipped(grads, work, max_norm, want)
        if max_norm == 1e9:
            assert all(torch.equal(a, b) for a, b in zip(grads, work))


@pytest.mark.parametrize("dt,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F64, F64)],
                         ids=IDS)
@pytest.mark.parametrize("offset", [0, 1, 3, 5])
@pytest.mark.parametrize("more", [[], [1_500_001, 3, 600_000]], ids=["one launch", "two"])
def test_out_of_place_into_a_flat_buffer(dt, out, offset, more):
    """Ragged sizes, so the flat buffer's parts start anywhere; the source too."""
    sizes = [9, 4096, 31, 1, 100001, 8, 2048, 77] + more
    grads = grads_of(sizes, dt, offset=offset)
    kept = [g.clone() for g in grads]
    flat = torch.full((sum(sizes) + 2,), 7.0, device="cuda", dtype=out)
    outs = list(flat[1:-1].split(sizes))
    for max_norm in (0.5, 1e9):
        norm = binding.msda_clip_grad_norm(binding.GradientBuffers(grads, out=outs), max_norm)
        check_clipped(grads, outs, max_norm, check_norm(norm, grads, 2.0))
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))
        assert flat[0] == 7 and flat[-1] == 7


def test_mixed_types():
    grads = [t for dt in (F32, BF16, F64, F16) for t in grads_of([1000, 3, 70001], dt, seed=dt.itemsize)]
    work = [g.clone() for g in grads]
    norm = binding.msda_clip_grad_norm(work, 0.1)
    check_clipped(grads, work, 0.1, check_norm(norm, grads, 2.0))
    check_norm(binding.msda_grad_norm(grads, math.inf), grads, math.inf)


def test_more_tensors_than_one_table_holds():
    grads = grads_of([(i * 37) % 301 for i in range(2500)], F32)
    work = [g.clone() for g in grads]
    norm = binding.msda_clip_grad_norm(work, 0.1)
    check_clipped(grads, work, 0.1, check_norm(norm, grads, 2.0))


@pytest.mark.parametrize("dt", [F32, BF16], ids=IDS)
@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-19, 1e17, 1e19, 1e30])
def test_squares_past_fp32s_range(dt, size):
    """Entries whose squares (or their sum) overflow or vanish in fp32."""
    for n in (5000, 2_000_003):
        grads = grads_of([n, 17, 1], dt, scale=size)
        norm = binding.msda_grad_norm(grads)
        check_norm(norm, grads, 2.0)
        mixed = grads_of([n], dt, scale=size) + grads_of([n], dt, seed=1, scale=1.0)
        check_norm(binding.msda_grad_norm(mixed), mixed, 2.0)


def test_zeros():
    grads = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]
    norm = binding.msda_clip_grad_norm(grads, 0.1)
    assert float(norm) == 0 and not any(g.any() for g in grads)
    assert float(binding.msda_grad_norm([torch.empty(0, device="cuda")])) == 0
    assert float(binding.msda_clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0
    assert float(binding.msda_grad_norm([])) == 0


@pytest.mark.parametrize("dt", [F32, BF16, F16, F64], ids=IDS)
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("at", [0, 3000, 4999])
def test_entries_that_are_not_finite(dt, kind, at):
    for value, more in [(v, m) for v in (float("inf"), float("-inf"), float("nan")) for m in (70, 3_000_001)]:
        grads = grads_of([5000, more], dt)
        grads[0][at] = value
        norm = binding.msda_clip_grad_norm(grads, 0.1, kind)
        if value != value:
            assert norm.isnan() and all(g.isnan().all() for g in grads)
        else:
            assert float(norm) == math.inf
            assert grads[0][at].isnan()
            keep = torch.arange(5000, device="cuda") != at
            assert not grads[0][keep].any() and not grads[1].any()


def test_same_bits_again():
    grads = grads_of([1000, 3, 900001, 70], BF16)
    norms = {float(binding.msda_grad_norm(grads)) for _ in range(5)}
    assert len(norms) == 1
    buf = binding.GradientBuffers(grads, out=[torch.empty(g.shape, device="cuda") for g in grads])
    assert float(binding.msda_clip_grad_norm(buf, 0.1)) in norms


def test_offsets_past_32_bits():
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[0], g[n // 2], g[-1] = 3.0, 4.0, 12.0
    assert float(binding.msda_grad_norm([g])) == 13.0
    assert float(binding.msda_grad_norm([g], math.inf)) == 12.0
    out = torch.full((n,), 5.0, device="cuda")
    binding.msda_clip_grad_norm(binding.GradientBuffers([g], out=[out]), 1.0)
    f = 1.0 / (13.0 + 1e-6)
    for at, v in ((0, 3.0), (n // 2, 4.0), (n - 1, 12.0)):
        assert abs(float(out[at]) - v * f) <= 40 * U32 * v * f
    assert int(out.count_nonzero()) == 3


def test_buffers_follow_their_tensors():
    grads = grads_of([1000, 500], F32)
    buf = binding.GradientBuffers(grads)
    first = float(binding.msda_grad_norm(buf))
    for g in grads:
        g.mul_(2)
    assert abs(float(binding.msda_grad_norm(buf)) - 2 * first) <= 70 * U32 * first
    # the caller's objects may change; the buffers keep the memory they were given
    held = grads[0]
    held.data = torch.ones(7, device="cuda")
    assert abs(float(binding.msda_grad_norm(buf)) - 2 * first) <= 70 * U32 * first
    # a storage freed behind the buffers' back is noticed
    grads[1].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="resized"):
        binding.msda_grad_norm(buf)


def test_dense_tensors_of_any_order():
    w = grads_of([4 * 8 * 3 * 3], F32)[0].view(4, 8, 3, 3).contiguous(memory_format=torch.channels_last)
    t = grads_of([35], F32, seed=1)[0].view(5, 7).t()
    before = [w.clone(), t.clone()]
    norm = binding.msda_clip_grad_norm([w, t], 0.1)
    check_clipped(before, [w, t], 0.1, check_norm(norm, before, 2.0))


def test_clip_grad_norm_of_parameters():
    ps = [torch.nn.Parameter(torch.zeros(s, device="cuda")) for s in ((3, 5), (7,), (2, 2))]
    ps[0].grad, ps[1].grad = torch.randn(3, 5, device="cuda"), torch.randn(7, device="cuda")
    before = [ps[0].grad.clone(), ps[1].grad.clone()]
    norm = binding.clip_grad_norm_(iter(ps), 0.1)
    check_clipped(before, [ps[0].grad, ps[1].grad], 0.1, check_norm(norm, before, 2.0))
    assert ps[2].grad is None
    norm = binding.clip_grad_norm_(ps[1], 1e9)
    assert float(binding.clip_grad_norm_([ps[2]], 1.0)) == 0
    ps[0].grad[1, 1] = float("nan")
    kept = ps[1].grad.clone()
    with pytest.raises(RuntimeError, match="nan"):
        binding.clip_grad_norm_(ps, 0.1, error_if_nonfinite=True)
    assert torch.equal(ps[1].grad, kept)


def test_autograd_sees_the_change_in_place():
    x = torch.ones(8, device="cuda", requires_grad=True)
    g = torch.ones(8, device="cuda")
    y = (x * g).sum()                    # saves g
    binding.msda_clip_grad_norm([g], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_another_stream_and_captured_graphs():
    a, b = grads_of([5000, 3_000_001, 3], BF16), grads_of([300] * 20, F32, seed=2)
    oa = [torch.empty(g.shape, device="cuda") for g in a]
    ob = [torch.empty_like(g) for g in b]
    A, B = binding.GradientBuffers(a, out=oa), binding.GradientBuffers(b, out=ob)
    na, nb = binding.msda_clip_grad_norm(A, 0.1), binding.msda_clip_grad_norm(B, 0.1)
    want = [t.clone() for t in (na, nb, *oa, *ob)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm = binding.msda_clip_grad_norm(A, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(norm, want[0])
    graphs, norms = [], []
    for buf in (A, B):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(binding.msda_clip_grad_norm(buf, 0.1))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for t in (*norms, *oa, *ob):
            t.fill_(3.0)
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*norms, *oa, *ob), want))
    a[0].mul_(100)                        # a replay follows its inputs
    graphs[0].replay()
    torch.cuda.synchronize()
    check_norm(norms[0], a, 2.0)


def test_refusals():
    g = torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        binding.msda_grad_norm([g.cpu()])
    with pytest.raises(ValueError, match="unsupported dtype"):
        binding.msda_grad_norm([g.int()])
    with pytest.raises(ValueError, match="dense"):
        binding.msda_grad_norm([g[::2]])
    with pytest.raises(ValueError, match="sparse"):
        binding.msda_grad_norm([g.to_sparse()])
    with pytest.raises(ValueError, match="share memory"):
        binding.msda_grad_norm([g, g])
    with pytest.raises(ValueError, match="share memory"):
        binding.msda_clip_grad_norm([g[:5], g[4:]], 1.0)
    with pytest.raises(ValueError, match="share memory"):
        binding.GradientBuffers([g.half()], out=[g]) and binding.GradientBuffers([g[:4]], out=[g[2:6]])
    with pytest.raises(ValueError, match="norm_type"):
        binding.msda_grad_norm([g], 1.0)
    with pytest.raises(ValueError, match="outputs for"):
        binding.GradientBuffers([g], out=[])
    with pytest.raises(ValueError, match="shape"):
        binding.GradientBuffers([g], out=[torch.empty(9, device="cuda")])
    with pytest.raises(ValueError, match="output of"):
        binding.GradientBuffers([g], out=[torch.empty(8, device="cuda", dtype=F16)])
    for bad in (-1.0, float("nan")):
        with pytest.raises(binding.MSDAError, match="SHAPE"):
            binding.msda_clip_grad_norm([g], bad)
    assert torch.equal(g, torch.ones(8, device="cuda"))


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_accesses_stay_in_bounds(offset):
    binding.use_library(build.CHECKED_LIBRARY)
    try:
        for dt in (F32, BF16, F64):
            for sizes in SIZES:
                grads = grads_of(sizes, dt, offset=offset)
                work = [g.clone() for g in grads]
                norm = binding.msda_clip_grad_norm(work, 0.1)
                check_clipped(grads, work, 0.1, check_norm(norm, grads, 2.0))
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()
