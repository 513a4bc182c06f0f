"""Attention's range of scales, checked on the host: what times log2(e) is an fp32 number."""
import pytest

from test_attention_host import bwd, dims, fwd, so  # noqa: F401


@pytest.mark.parametrize("call", [fwd, bwd])
def test_scales(so, call):  # noqa: F811
    for scale in (2.4e38, 3e38, 3.4e38):
        assert call(so, dims(), scale=scale) == 2
    for scale in (0.0, 1e-40, 2.3e38):               # reaches the workspace's check
        assert call(so, dims(), scale=scale, mask=0x10000, ws=None) == 5
