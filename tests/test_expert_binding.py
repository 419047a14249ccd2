"""The binding of the expert operators, without a GPU: orders of nothing."""
import pytest

from block_scaled_fp8_x1_gb300 import ops


def test_an_order_of_no_experts_is_refused():
    with pytest.raises(ValueError, match="0 experts"):
        ops._divided(256, 0, "codes W")
    with pytest.raises(ValueError, match="3 experts"):
        ops._divided(256, 3, "codes W")
    assert ops._divided(256, 2, "codes W") == 128
