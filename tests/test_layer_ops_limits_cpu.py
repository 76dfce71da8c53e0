"""Bounds of the attention call's sizes and scalars, before any device is touched.  A call that passes them here stops
at its missing workspace."""
import pytest

from fp8_dynamic_scaled_b200 import binding as b
from test_layer_ops_cpu import INV, P, attend


def sized(tokens, heads, kv_heads, max_q):
    w = heads * 64
    return attend(tokens=tokens, heads=heads, kv_heads=kv_heads, cu=P, max_q=max_q, ldq=w, ldo=w, ws=None)


@pytest.mark.parametrize("kv_heads", [1, 2, 1024])
def test_rows_that_int32_cannot_count(kv_heads):
    assert sized(1 << 20, 1 << 16, kv_heads, 1 << 20) == INV                 # 2^36 rows
    assert sized(1 << 15, 1 << 16, kv_heads, 1 << 15) == INV                 # 2^31
    assert sized((1 << 15) - 1, 1 << 16, kv_heads, (1 << 24) - 1) == b.FP8_ERR_WORKSPACE      # the most; a loose bound
    assert sized((1 << 31) - 1, 1 << 16, kv_heads, 16) == b.FP8_ERR_WORKSPACE
    assert sized((1 << 31) - 1, 1 << 16, kv_heads, 1 << 15) == INV


def test_softmax_scale_times_log2e_is_finite():
    for scale in (2.359e38, 3.4e38, float("nan")):
        assert attend(scale=scale, ws=None) == INV and attend(scale=-scale, ws=None) == INV
    for scale in (2.3586e38, -2.3586e38, 2.0 ** 90, 0.0):
        assert attend(scale=scale, ws=None) == b.FP8_ERR_WORKSPACE
