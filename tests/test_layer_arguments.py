"""What MultiHeadAttention is made with is checked when it is made."""
import pytest

from scale_deformable_attention_msda_gb300.layer import MultiHeadAttention


@pytest.mark.parametrize("kw", [dict(dim=60, num_heads=5), dict(dim=512, num_heads=2), dict(dim=32, num_heads=8), dict(dim=256, num_heads=0),
                                dict(dim=256, num_heads=8, kv_heads=0), dict(dim=256, num_heads=8, kv_heads=-8), dict(dim=256, num_heads=-8),
                                dict(dim=0, num_heads=8), dict(dim=256, num_heads=4, kv_heads=8)], ids=str)
def test_refused(kw):
    with pytest.raises(ValueError):
        MultiHeadAttention(**kw)


@pytest.mark.parametrize("kw", [dict(dim=8, num_heads=1), dict(dim=128, num_heads=1), dict(dim=1024, num_heads=8, kv_heads=1),
                                dict(dim=72, num_heads=3)], ids=str)
def test_made(kw):
    layer = MultiHeadAttention(**kw)
    assert layer.head_dim * layer.num_heads == layer.dim
