"""The row statistics r = 1/sqrt(mean(v^2) + eps) of residual_norm, to the last bit.

Rows of integers of at most 32 and a power of two of columns: every partial sum of squares is an
integer of at most 2^23, the mean a multiple of 2^-13 up to 2^10, and with an eps of such a form the
argument of the root is exact in FP32.  What is left is the root: the Newton step's own error is 3/8 of
the square of the hardware root's (2^-21 at most: 2^-43), so the one rounding of the result is half a
unit in the last place, and 2^-10 of a unit covers the rest.
"""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu


def ulps(r, exact):
    """|r - exact| in units in the last place of exact."""
    step = torch.exp2(torch.floor(torch.log2(exact)) - 23)
    return float(((r.double() - exact).abs() / step).max())


@pytest.mark.parametrize("K", [128, 512, 1024, 4096, 8192])
@pytest.mark.parametrize("eps", [0.0, 0.125, 3.0, 700.0])
def test_rounded_once(fp8lib, K, eps):
    M = 2000
    gen = torch.Generator("cuda").manual_seed(K)
    draw = lambda: torch.randint(-32, 33, (M, K), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    h, y, one = draw(), draw(), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    h[0], y[0, 1:] = 0.0, 0.0
    h[0, 0], y[0, 0] = 3.0, 5.0
    r = fp8lib.residual_norm(h, torch.zeros_like(h), one, eps, emit="bf16")
    assert torch.equal(r.h, h)
    assert ulps(r.r_pre, ref.rstd(h.double(), eps)) <= 0.5 + 2.0 ** -10
    r = fp8lib.residual_norm(h, y, one, eps, post_gamma=one, emit="fp8")
    assert ulps(r.r_post, ref.rstd(y.double(), eps)) <= 0.5 + 2.0 ** -10
