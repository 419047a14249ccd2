"""Groups ranked by sums of two whose biases cancel.

The sum of two is small and each of the two was rounded at the size of its bias: the order of the groups is
still that of the exact sums wherever these are 2^-40 apart, or 2^-44 of the largest |score + bias|."""
import numpy as np
import pytest
import torch

import expert_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def group_sums(z, bias, G, score):
    v = ref.scores(z, score) + bias
    return np.sort(v.reshape(len(z), G, -1), axis=2)[:, :, -2:].sum(2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,top", [(16, 4, 2), (24, 8, 3), (256, 8, 4), (96, 4, 1)])
@pytest.mark.parametrize("B", [16.0, 100.0, 1000.0])
def test_sums_that_cancel(fp8lib, B, E, G, top, score):
    r = np.random.default_rng(E + int(B))
    T, gs = 1500, E // G
    z = (0.3 + r.uniform(2e-6, 2e-5, (T, 1)) * r.standard_normal((T, E))).astype(np.float32)
    bias = np.full(E, -3.0 * B, np.float32)
    for g in range(G):
        first, second = r.permutation(gs)[:2]
        bias[g * gs + first], bias[g * gs + second] = B, -B
    # rows whose border the definition itself can tell in 64 bits, and the router's pairs too
    order = np.sort(group_sums(z.astype(np.float64), bias.astype(np.float64), G, score), axis=1)
    clear = order[:, G - top] - order[:, G - top - 1] > max(2.0 ** -39, 2.0 ** -44 * B)
    assert clear.mean() > 0.9
    z = z[clear]
    # as many experts as groups: the one with the positive bias of every group that is kept
    got = fp8lib.route_topk(torch.tensor(z, device=DEV), top, score=score, bias=torch.tensor(bias, device=DEV), n_groups=G,
                            top_groups=top, group_rank=2).index.cpu().numpy()
    _, want = ref.route(z, top, score, bias, n_groups=G, top_groups=top, group_rank=2)
    assert np.array_equal(np.sort(got, 1), np.sort(want, 1))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), 3e38])
def test_biases_without_bound(fp8lib, bad):
    """An infinite or huge bias in one group leaves the order of the others alone."""
    r = np.random.default_rng(1)
    z = r.standard_normal((200, 64)).astype(np.float32)
    bias = (0.1 * r.standard_normal(64)).astype(np.float32)
    bias[3], bias[4] = bad, 0.5 * bad
    got = fp8lib.route_topk(torch.tensor(z, device=DEV), 6, score="sigmoid", bias=torch.tensor(bias, device=DEV), n_groups=8,
                            top_groups=3, group_rank=2).index.cpu().numpy()
    _, want = ref.route(z, 6, "sigmoid", bias, n_groups=8, top_groups=3, group_rank=2)
    assert np.array_equal(got, want)
