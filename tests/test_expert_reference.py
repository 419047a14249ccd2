"""The 64-bit definitions of the expert-layer tests, against torch's autograd and hand-made cases."""
import numpy as np
import pytest
import torch

import expert_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_and_its_gradient(score, renorm):
    torch.manual_seed(1)
    z = torch.randn((5, 12), dtype=torch.float64, requires_grad=True)
    w, i = ref.route(z.detach().numpy(), 3, score, renormalize=renorm, scale=2.0)
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    top = torch.topk(s, 3, dim=1)
    t = top.values / top.values.sum(1, keepdim=True) if renorm else top.values
    assert np.array_equal(i, top.indices.numpy()) and np.allclose(w, 2.0 * t.detach().numpy(), rtol=1e-14)
    g = torch.randn((5, 3), dtype=torch.float64)
    (2.0 * t * g).sum().backward()
    assert np.allclose(ref.route_bwd(g.numpy(), z.detach().numpy(), i, score, renorm, 2.0), z.grad.numpy(), rtol=1e-12, atol=1e-15)


def test_route_groups_by_hand():
    z = np.array([[0.0, 3.0, 2.0, 2.0, 1.0, 1.0]])
    _, i = ref.route(z, 2, n_groups=3, top_groups=1, group_rank=1)
    assert i.tolist() == [[1, 0]]
    _, i = ref.route(z, 3, "sigmoid", np.zeros(6), n_groups=3, top_groups=2, group_rank=2)
    assert i.tolist() == [[2, 3, 4]] or i.tolist() == [[1, 2, 3]]
    z[0, :] = -np.inf
    w, i = ref.route(z, 2)
    assert (i == -1).all() and (w == 0).all()


def test_rows_by_hand():
    pos, src, start, count = ref.rows(np.array([[1, 0], [1, 2], [-1, 1]]), 3, 1)
    assert src.tolist() == [1, 0, 2, 5, 3, -1] and start.tolist() == [0, 1, 4, 5] and count.tolist() == [1, 3, 1]
    assert pos.tolist() == [[1, 0], [2, 4], [-1, 3]]
    _, src, start, _ = ref.rows(np.array([[1], [1]]), 3, 128)
    assert start.tolist() == [0, 0, 128, 128] and src[:3].tolist() == [0, 1, -1] and len(src) == 256


def test_e4m3_values():
    q = torch.arange(256, dtype=torch.uint8)
    want = q.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.decode_e4m3(q.numpy()), want, equal_nan=True)
