"""The 64-bit definitions of the block operators against differences (CPU)."""
import pytest
import torch

import block_reference as ref


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_residual_norm_gradients_against_differences(post, gated):
    gen = torch.Generator().manual_seed(3 + 2 * post + gated)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    M, K, eps, alpha = 5, 24, 1e-3, 0.7
    v = {"h": rnd(M, K), "y": rnd(M, K), "pre": 1 + 0.3 * rnd(K)}
    if post:
        v["post"] = 1 + 0.3 * rnd(K)
    if gated:
        v["gate"] = rnd(K)
    dz, dh = rnd(M, K), rnd(M, K)

    def loss(v):
        h2, z, _, _ = ref.residual_norm(v["h"], v["y"], v["pre"], eps, v.get("post"), v.get("gate"), alpha)
        return float((z * dz).sum() + (h2 * dh).sum())

    h2, _, r, rp = ref.residual_norm(v["h"], v["y"], v["pre"], eps, v.get("post"), v.get("gate"), alpha)
    g = ref.residual_norm_bwd(dz, dh, h2, v["y"], v["pre"], r, v.get("post"), rp, v.get("gate"), alpha)
    grads = {"h": g["dh"][0], "y": g["dy"][0], "pre": g["dpre"][0]}
    if post:
        grads["post"] = g["dpost"][0]
    if gated:
        grads["gate"] = g["dgate"][0]
    assert set(grads) == set(v)
    step = 1e-5
    for name, x in v.items():
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        diff = (loss({**v, name: x + step * d}) - loss({**v, name: x - step * d})) / (2 * step)
        want = float((grads[name] * d).sum())
        # central differences: step^2 of truncation, 1e-16 / step of rounding, on sums of ~10
        assert abs(diff - want) <= 1e-7 * (1 + abs(want)), name
