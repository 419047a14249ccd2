"""matvec_nvfp4 where the sums in units of the row scale would leave FP32's range and the result does
not: the row scale is the weights' largest magnitude / 2688, so that those sums are up to 2688
times the result over that magnitude.

Bounds as for ordinary sizes: one BF16 rounding (half a subnormal step, 2^-134, beside it) and
(32 + K / 128) 2^-22 of the terms' magnitudes; sums below 2^-126 add FP32's subnormal half steps,
fewer than 64 of 2^-150, twice that after the row scale's last factor: 2^-133 covers all of it."""
import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 3, 9])
@pytest.mark.parametrize("x_size,w_size", [(1e36, 0.02), (5e36, 1e-6), (1e37, 1e-25), (1e20, 1e15), (1e-12, 1e25), (1e-36, 1e33), (1e-30, 1e-3)])
def test_range(fp8lib, M, x_size, w_size):
    N, K = 256, 1024
    w = (synth.normal_bf16((N, K), 1.0, 3, "cuda").double() * w_size).to(torch.bfloat16)
    w[N // 2] = 0.0
    w = fp8lib.quantize_nvfp4(w)
    x = (synth.normal_bf16((M, K), 1.0, 4, "cuda").double() * x_size).to(torch.bfloat16)
    wd = ref.decode_nvfp4(*w)
    assert bool(torch.isfinite(wd).all()) and float(wd.abs().max()) > 0
    want, mag = x.double() @ wd.t(), x.double().abs() @ wd.abs().t()
    assert float(want.abs().max()) < 3e38
    for splits in (0, 1, 3):
        y = fp8lib.matvec_nvfp4(x, *w, splits=splits)
        bad = ~((y.double() - want).abs() <= ref.BF16_HALF * want.abs() + (32 + K / 128) * 2.0 ** -22 * mag + 2.0 ** -133)
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("M", [1, 4, 12])
def test_every_size_of_row_scale(fp8lib, M):
    """Small integers times powers of two: every sum is exact, whatever the row scale's exponent."""
    N, K = 256, 512
    gen = torch.Generator("cuda").manual_seed(2)
    q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sf = torch.full((fp8lib.nvfp4_scale_bytes(N, K),), 56, dtype=torch.uint8, device="cuda")   # E4M3 1
    g = 1.5 * torch.exp2(torch.linspace(-125, 100, N, device="cuda").round())
    x = torch.randint(-4, 5, (M, K), generator=gen, device="cuda").to(torch.bfloat16)
    sums = x.double() @ ref.decode_nvfp4(q, sf, torch.ones_like(g)).t()
    want = (sums * g.double()).float().to(torch.bfloat16)     # the product has 24 bits or fewer
    assert torch.equal(fp8lib.matvec_nvfp4(x, q, sf, g), want)
