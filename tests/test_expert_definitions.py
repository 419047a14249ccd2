"""Definitions of the expert operators that allow one answer, and the most rows an order can need."""
import itertools

import numpy as np
import pytest

import expert_reference as ref


def test_groups_by_their_two_best():
    """Sigmoid scores of 0, 3 | 2, 2 | 1, 1: sums 1.4526, 1.7616, 1.4621, so the last two groups are kept; by their
    single best (0.9526, 0.8808, 0.7311) the first two."""
    z = np.array([[0.0, 3.0, 2.0, 2.0, 1.0, 1.0]])
    _, i = ref.route(z, 3, "sigmoid", np.zeros(6), n_groups=3, top_groups=2, group_rank=2)
    assert i.tolist() == [[2, 3, 4]]
    _, i = ref.route(z, 3, "sigmoid", np.zeros(6), n_groups=3, top_groups=2, group_rank=1)
    assert i.tolist() == [[1, 2, 3]]
    _, i = ref.route(z, 4, "sigmoid", np.array([0.0, 0, 0, 0, 0.2, 0.2]), n_groups=3, top_groups=2, group_rank=2)
    assert i.tolist() == [[4, 5, 2, 3]]


def most_rows(P, E, align):
    """The largest sum of the experts' counts, each rounded up, over every way to share P pairs among at most E
    experts: an expert at a time, the best of every size of its share."""
    best = [0] + [-1] * P                # pairs given away -> rows, for the experts so far
    for _ in range(min(E, P)):
        best = [max(best[p - c] + -(-c // align) * align for c in range(p + 1) if best[p - c] >= 0) for p in range(P + 1)]
    return best[P]


@pytest.mark.parametrize("align", [1, 128])
def test_capacity_is_the_most_that_an_order_can_need(align):
    from block_scaled_fp8_x1_gb300 import _abi, build_library
    build_library()
    f = _abi.lib().fp8rl_expert_rows_capacity
    for T, k, E in [*itertools.product((1, 2, 5), (1, 3), (1, 2, 4, 8)), (127, 1, 2), (64, 2, 3), (129, 1, 2), (86, 3, 3), (128, 2, 4),
                    (300, 1, 5)]:
        most = most_rows(T * k, E, align)
        assert f(T, k, E, align) == most == ref.capacity(T, k, E, align), (T, k, E)
