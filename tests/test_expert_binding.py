"""The binding of the expert operators, without a GPU: orders as trees of tensors, orders of nothing."""
import pytest
import torch
import torch.utils._pytree as pytree

from block_scaled_fp8_x1_gb300 import ops


def arrays():
    return [torch.arange(n, dtype=torch.int32) for n in (6, 6, 4, 3)]


@pytest.mark.parametrize("kind", [ops.ExpertRows, ops._SortedRows])
def test_an_order_is_a_tree_of_its_arrays(kind):
    """What moves, saves or counts the tensors of a structure finds those of an order, whoever made it."""
    rows = kind(*arrays(), 128)
    leaves, spec = pytree.tree_flatten({"rows": rows})
    assert [id(t) for t in leaves[:4]] == [id(t) for t in rows[:4]] and leaves[4] == 128
    moved = pytree.tree_map(lambda t: t.clone() if isinstance(t, torch.Tensor) else t, rows)
    assert isinstance(moved, ops.ExpertRows) and moved.align == 128
    for a, b in zip(moved[:4], rows[:4]):
        assert a is not b and torch.equal(a, b)
    assert getattr(moved, "layout", None) is None       # of the arrays that it was made from
    back = pytree.tree_unflatten(leaves, spec)["rows"]
    assert pytree.tree_flatten({"rows": back})[1] == spec


def test_an_order_of_no_experts_is_refused():
    with pytest.raises(ValueError, match="0 experts"):
        ops._divided(256, 0, "codes W")
    with pytest.raises(ValueError, match="3 experts"):
        ops._divided(256, 3, "codes W")
    assert ops._divided(256, 2, "codes W") == 128
