"""route_topk_bwd where scores end: logits far from zero, chosen scores next to nothing.

The sigmoid's derivative is s (1 - s).  Bound: the scores' and the exponential's FP32 roundings and the sum of
k weights, 2^-16 of (the largest |gradient of a weight| over the sum) times s (1 - s), each in 64 bits; half
a step of the result's type on top."""
import numpy as np
import pytest
import torch

import expert_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def np64(t):
    return t.detach().double().cpu().numpy()


def slope(z):
    """s (1 - s) with all its digits."""
    e = np.exp(-np.abs(z))
    return e / (1.0 + e) ** 2


def bwd_sigmoid(dw, z, index, renorm, scale):
    """route_bwd of the definitions with the derivative formed without a difference from 1."""
    g = dw * scale
    s = 1.0 / (1.0 + np.exp(-z))
    d = np.zeros_like(z)
    for t in range(z.shape[0]):
        p = s[t, index[t]]
        total = p.sum() + ref.TINY
        ds = (g[t] - (g[t] * p).sum() / total) / total if renorm else g[t]
        np.add.at(d[t], index[t], ds)
    return slope(z) * d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [8, 60, 200, 1000])
def test_sigmoid_of_large_logits(fp8lib, E, renorm, dtype):
    gen = torch.Generator(DEV).manual_seed(E)
    T, k = 24, 4
    at = torch.tensor([12.0, -12.0, 16.0, -16.0, 17.0, 20.0, -20.0, 40.0], device=DEV)
    z = (at.repeat(E // 8 + 1)[:E] + torch.randn((T, E), generator=gen, device=DEV)).to(dtype)
    index = torch.stack([torch.randperm(E, generator=gen, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    dw = torch.randn((T, k), generator=gen, device=DEV)
    got = np64(fp8lib.route_topk_bwd(dw, z, index, score="sigmoid", renormalize=renorm, scale=1.5))
    z64, i = np64(z), index.cpu().numpy()
    want = bwd_sigmoid(np64(dw), z64, i, renorm, 1.5)
    s = 1.0 / (1.0 + np.exp(-z64))
    total = np.take_along_axis(s, i, 1).sum(1, keepdims=True) if renorm else 1.0
    size = 4 * 1.5 * np.abs(np64(dw)).max(1, keepdims=True) / total * slope(z64)
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= half * np.abs(want) + 2.0 ** -16 * size)


def test_sigmoid_ends_in_zero_not_in_nan(fp8lib):
    inf = float("inf")
    z = torch.tensor([[-inf, inf, 200.0, -200.0, torch.finfo(torch.float32).max, torch.finfo(torch.float32).min, 0.0]], device=DEV)
    index = torch.arange(7, dtype=torch.int32, device=DEV)[None]
    d = fp8lib.route_topk_bwd(torch.ones((1, 7), device=DEV), z, index, score="sigmoid", renormalize=False)
    assert d.tolist() == [[0.0] * 6 + [0.25]]


@pytest.mark.parametrize("below", [20.0, 35.0, 46.0, 48.0, 60.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_chosen_scores_next_to_nothing(fp8lib, score, below):
    """A bias can choose experts whose scores are `e^-below` of the row's: where their sum is no longer far above
    the 1e-20 that is added to it, the weights do change with the scores of all experts.

    Bound: s_e (|ds_e| + sum s |ds|), the magnitudes that are added, times 2^-16: FP32 scores at a distance of
    `below` are within 2^-18 of themselves."""
    T, E, k = 16, 40, 3
    gen = torch.Generator(DEV).manual_seed(int(below))
    z = torch.randn((T, E), generator=gen, device=DEV)
    z[:, :10] -= below
    index = torch.stack([torch.randperm(10, generator=gen, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    dw = 1.0 + torch.rand((T, k), generator=gen, device=DEV)
    got = np64(fp8lib.route_topk_bwd(dw, z, index, score=score, scale=1.5))
    z64, i = np64(z), index.cpu().numpy()
    want = ref.route_bwd(np64(dw), z64, i, score, True, 1.5)
    s = ref.scores(z64, score)
    p = np.take_along_axis(s, i, 1)
    total = p.sum(1, keepdims=True) + ref.TINY
    ds = np.zeros((T, E))
    np.put_along_axis(ds, i, 1.5 * (np64(dw) + (np64(dw) * p).sum(1, keepdims=True) / total) / total, 1)
    size = s * (ds + (s * ds).sum(1, keepdims=True))
    assert np.all(np.abs(got - want) <= 2.0 ** -16 * size)
