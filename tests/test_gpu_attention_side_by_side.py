"""Attention's forward and backward passes of several kinds on several streams at once: blocks
of different kernels share SMs and their tensor memory, and no result changes."""
import pytest
import torch

from scale_deformable_attention_msda_gb300 import binding
from test_gpu_attention import BF16, F16, F32, _lib, make_mask, operands  # noqa: F401

pytestmark = pytest.mark.gpu


def test_steps_on_four_streams():
    kinds = [((2, 300, 300, 8, 8, 32), BF16, "heads"), ((1, 1024, 1024, 4, 2, 64), F16, "none"), ((1, 600, 700, 4, 1, 128), BF16, "padding"),
             ((4, 60, 900, 4, 4, 32), F16, "pairs"), ((2, 1, 4000, 8, 2, 64), F16, "none"), ((2, 200, 200, 4, 4, 32), F32, "none")]
    cases = []
    for i, (sizes, dt, kind) in enumerate(kinds):
        q, k, v, go, gen = operands(*sizes, dt, seed=i)
        cases.append((q, k, v, go, make_mask(kind, sizes[0], sizes[3], sizes[1], sizes[2], gen)))

    def step(q, k, v, go, mask):
        out, lse, rest = binding.msda_attention_forward(q, k, v, mask=mask, rest=True)
        return [out, lse, *binding.msda_attention_backward(go, q, k, v, out, lse, mask=mask, rest=rest)]
    want = [step(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for turn in range(12):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[(turn + i) % 4]):
                got.append((i, step(*c)))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(want[i], g)), kinds[i]
    assert binding.msda_device_check() == 0
