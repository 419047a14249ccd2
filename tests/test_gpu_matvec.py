"""y = x W^T for a few BF16 tokens on NVFP4 weights, on the GPU, against the 64-bit product.

The products are exact.  A sum chains 8 MMA additions inside 128 elements of K (each adds 16
products, aligned to the largest: 2^-22 of the terms' magnitudes allowed for one), then at most
K / 128 + 16 FP32 additions: (32 + K / 128) 2^-22 of the sum of the terms' magnitudes.  An element
below 2^-28 of the largest of its 128 neighbours loses at most 2^-39 of that one, which the same
bound covers where the row's weights are of one size, as here.  One BF16 rounding (2^-8) follows.
"""
import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu


def weights(fp8lib, N, K, seed=3):
    w = synth.normal_bf16((N, K), 0.02, seed, "cuda")
    w[N // 2] = 0.0                                   # a zero row: all scales zero
    return fp8lib.quantize_nvfp4(w)


def check(y, x, w):
    wd = ref.decode_nvfp4(*w)
    K = x.shape[1]
    want = x.double() @ wd.t()
    mag = x.double().abs() @ wd.abs().t()
    bound = ref.BF16_HALF * want.abs() + (32 + K / 128) * 2.0 ** -22 * mag
    bad = ~((y.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"


@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (1, 3584, 3584), (2, 256, 512), (3, 128, 768), (5, 4608, 3584), (7, 640, 1280),
                                   (8, 3584, 3584), (9, 384, 256), (11, 3584, 18944), (16, 512, 18944), (1, 37888, 3584),
                                   (16, 37888, 3584), (1, 128, 65536), (16, 128, 65536)])
def test_product(fp8lib, M, N, K):
    x = synth.normal_bf16((M, K), 1.0, M + K, "cuda", outlier_channels=2, outlier_scale=30.0)
    if M > 2:
        x[1] = 0.0
    w = weights(fp8lib, N, K)
    y = fp8lib.matvec_nvfp4(x, *w)
    check(y, x, w)
    assert torch.equal(y, fp8lib.matvec_nvfp4(x, *w))
    assert float(y[:, N // 2].abs().max()) == 0.0
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("M", [1, 6, 13])
@pytest.mark.parametrize("splits", range(1, 9))
def test_every_split(fp8lib, M, splits):
    N, K = 640, 1792                                   # 14 blocks of 128: uneven shares
    x = synth.normal_bf16((M, K), 1.0, 5, "cuda")
    w = weights(fp8lib, N, K)
    y = fp8lib.matvec_nvfp4(x, *w, splits=splits)
    check(y, x, w)
    assert torch.equal(y, fp8lib.matvec_nvfp4(x, *w, splits=splits))


def test_every_token_count(fp8lib):
    N, K = 256, 1024
    w = weights(fp8lib, N, K)
    x = synth.normal_bf16((16, K), 1.0, 8, "cuda")
    for M in range(1, 17):
        check(fp8lib.matvec_nvfp4(x[:M], *w), x[:M], w)


def test_exact_products_of_exact_operands(fp8lib):
    """Small integers: every sum is exact, so every code, scale and position must be right."""
    N, K, M = 256, 2048, 4
    gen = torch.Generator("cuda").manual_seed(2)
    q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sf = torch.randint(0, 4, (fp8lib.nvfp4_scale_bytes(N, K),), generator=gen, device="cuda")
    sf = (sf * 8 + 48).to(torch.uint8)                 # E4M3 1/2, 1, 2, 4
    g = torch.exp2(torch.randint(-3, 3, (N,), generator=gen, device="cuda").float())
    x = torch.randint(-4, 5, (M, K), generator=gen, device="cuda").to(torch.bfloat16)
    want = (x.double() @ ref.decode_nvfp4(q, sf, g).t()).to(torch.bfloat16)
    for splits in (0, 1, 3, 8):
        assert torch.equal(fp8lib.matvec_nvfp4(x, q, sf, g, splits=splits), want)


@pytest.mark.parametrize("scale", [2.0 ** -130, 1e-30, 1e-6, 1e20, 1e33])
def test_size_of_x(fp8lib, scale):
    N, K = 256, 512
    w = weights(fp8lib, N, K)
    x = (synth.normal_bf16((3, K), 1.0, 4, "cuda").double() * scale).to(torch.bfloat16)
    y = fp8lib.matvec_nvfp4(x, *w)
    wd = ref.decode_nvfp4(*w)
    want, mag = x.double() @ wd.t(), x.double().abs() @ wd.abs().t()
    # half a step of subnormal results beside the usual bound
    assert bool(((y.double() - want).abs() <= ref.BF16_HALF * want.abs() + 36 * 2.0 ** -22 * mag + 2.0 ** -133).all())


def test_nan_and_infinity_stay_in_their_token(fp8lib):
    N, K = 256, 512
    w = weights(fp8lib, N, K)
    x = synth.normal_bf16((5, K), 1.0, 4, "cuda")
    want = fp8lib.matvec_nvfp4(x, *w)
    x[1, 7] = float("nan")
    x[3, 300] = float("inf")
    y = fp8lib.matvec_nvfp4(x, *w)
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any())
    for m in (0, 2, 4):
        assert torch.equal(y[m], want[m])


def test_strides_another_stream_and_capture(fp8lib):
    M, N, K = 6, 384, 768
    w = weights(fp8lib, N, K)
    x = synth.normal_bf16((M, K), 1.0, 4, "cuda")
    want = fp8lib.matvec_nvfp4(x, *w)
    wide = torch.full((2 * M, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[::2, 8:8 + K] = x
    buf = torch.zeros((M, N + 64), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8lib.matvec_nvfp4(wide[::2, 8:8 + K], *w, out=buf[:, 32:32 + N])
    side.synchronize()
    assert torch.equal(buf[:, 32:32 + N], want)
    assert float(buf[:, :32].abs().max()) == 0.0 and float(buf[:, 32 + N:].abs().max()) == 0.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fp8lib.matvec_nvfp4(x, *w)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, (want.float() * 2).to(torch.bfloat16))


def test_no_tokens(fp8lib):
    w = weights(fp8lib, 128, 256)
    assert fp8lib.matvec_nvfp4(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), *w).shape == (0, 128)


def test_more_accurate_than_quantizing_x(fp8lib):
    """What the 16-bit activation buys over the linear that quantizes it to 4 bits."""
    N, K, M = 1024, 3584, 8
    x = synth.normal_bf16((M, K), 1.0, 4, "cuda", outlier_channels=3, outlier_scale=30.0)
    wb = synth.normal_bf16((N, K), 0.015, 9, "cuda")
    w = fp8lib.quantize_nvfp4(wb)
    exact = x.double() @ wb.double().t()
    rel = lambda y: float((y.double() - exact).norm() / exact.norm())  # noqa: E731
    assert rel(fp8lib.matvec_nvfp4(x, *w)) < 0.9 * rel(fp8lib.linear_nvfp4(x, *w)[0])
