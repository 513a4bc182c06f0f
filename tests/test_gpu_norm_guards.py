"""What the layer norm's and the clipping's kernels write, and nothing beside it: every
output and the workspace between guard entries, through the C entries, in the normal and in
the range-checked build (whose report must stay clean)."""
import ctypes

import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding, build

pytestmark = pytest.mark.gpu

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
GUARD = 64                               # entries before and behind, a multiple of 16 bytes


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(params=["normal", "checked"])
def lib(request):
    so = binding.use_library(build.CHECKED_LIBRARY if request.param == "checked" else None)
    yield so
    try:
        assert binding.msda_device_check() == 0
    finally:
        binding.use_library()


class Guarded:
    """Tensors that start `offset` entries past a 16-byte boundary, each between guards; all
    NaN at first, which no result of these inputs is."""

    def __init__(self, offset=0):
        self.offset, self.held = offset, []

    def __call__(self, n, dt):
        flat = torch.full((n + 2 * GUARD + self.offset,), float("nan"), device="cuda", dtype=dt)
        self.held.append((flat, n))
        return flat[GUARD + self.offset:GUARD + self.offset + n]

    def check(self):
        for flat, n in self.held:
            assert flat[:GUARD + self.offset].isnan().all() and flat[GUARD + self.offset + n:].isnan().all()
            assert not flat[GUARD + self.offset:GUARD + self.offset + n].isnan().any()


# each form of the kernels, lengths that leave lanes idle, the last block's missing rows
SIZES = [(1, 1), (5, 7), (3, 8), (70, 40), (601, 256), (3001, 264), (33, 1000), (19, 1024), (9, 777), (1001, 33),
         (19, 4104), (7, 8191), (3, 8192), (3, 12001), (3, 13312), (2, 16384), (3, 32776)]


@pytest.mark.parametrize("dt,pdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F64, F64)], ids=str)
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("N,C", SIZES)
def test_layer_norm(lib, N, C, offset, dt, pdt):
    new = Guarded(offset)
    torch.manual_seed(N + C)

    def rows(n, t):
        return torch.randn(n + offset, device="cuda").to(t)[offset:]

    x, r, dy, ds, w, b = rows(N * C, dt), rows(N * C, dt), rows(N * C, dt), rows(N * C, dt), rows(C, pdt), rows(C, pdt)
    out, total, gx = new(N * C, dt), new(N * C, dt), new(N * C, dt)
    stats = F64 if dt == F64 else F32
    mean, rstd, gw, gb = new(N, stats), new(N, stats), new(C, pdt), new(C, pdt)
    dims = ctypes.byref(binding.msda_norm_dims_t(N, C))
    kinds = binding._DTYPES[dt], binding._DTYPES[pdt]
    stream = torch.cuda.current_stream().cuda_stream
    at = lambda t: t.data_ptr()          # noqa: E731
    assert lib.msda_layer_norm_forward(at(x), at(r), at(w), at(b), at(out), at(total), at(mean), at(rstd), 1e-5,
                                       dims, *kinds, stream) == 0
    need = lib.msda_layer_norm_backward_workspace_bytes(dims, kinds[0])
    space = torch.full((need + 2 * GUARD,), 77, device="cuda", dtype=torch.uint8)
    assert lib.msda_layer_norm_backward(at(dy), at(ds), at(x), at(r), at(w), at(mean), at(rstd), at(gx), at(gw), at(gb),
                                        at(space) + GUARD, need, dims, *kinds, stream) == 0
    torch.cuda.synchronize()
    new.check()
    assert (space[:GUARD] == 77).all() and (space[GUARD + need:] == 77).all()


@pytest.mark.parametrize("dt,to", [(F32, F32), (BF16, F32), (BF16, BF16), (F64, F64)], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("sizes", [[1, 7, 8, 9], [511, 513, 4097, 33], [100_003, 1, 70_001, 2_000_003]], ids=str)
def test_clipping(lib, sizes, offset, dt, to):
    new = Guarded(offset)
    torch.manual_seed(1)
    grads = [torch.randn(n + 5, device="cuda").to(dt)[5:] for n in sizes]
    outs = [new(n, to) for n in sizes]
    buf = binding.GradientBuffers(grads, out=outs)
    norm = torch.empty((), dtype=buf.norm_dtype, device="cuda")
    need = buf.workspace_bytes
    space = torch.full((need + 2 * GUARD,), 77, device="cuda", dtype=torch.uint8)
    assert lib.msda_clip_grad_norm(buf._ref, 0, 0.5, norm.data_ptr(), space.data_ptr() + GUARD, need,
                                   torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    new.check()
    assert (space[:GUARD] == 77).all() and (space[GUARD + need:] == 77).all()
