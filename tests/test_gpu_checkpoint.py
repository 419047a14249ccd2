"""SiLU-mul with an 8-bit checkpoint of its input, and the backward pass from it, on the GPU.

The forward's outputs are those of the separate operators bit for bit.  The backward is checked
in two ways: where the checkpoint decodes to BF16 numbers it must give the bits of the BF16
operator; otherwise every decoded element lies within the roundings of the 64-bit gradient: E4M3
half a step (2^-4 of the value, 2^-10 of the scale among the subnormals), BF16 half a step (2^-8 of
the value, 2^-134 among the subnormals, where a saturated gate's gradients lie), and 2^-16 of the
terms for the FP32 evaluation (its exponential and reciprocal included).
"""
import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu


def make(M, I, seed):
    gu = synth.normal_bf16((M, 2 * I), 1.5, seed, "cuda", outlier_channels=1, outlier_scale=30.0)
    dh = synth.normal_bf16((M, I), 1e-3, seed + 1, "cuda")
    gu[0, :I] = 0.0
    gu[M // 2, :] = 0.0                # zero groups in both halves
    gu[M - 1, :I] = 80.0               # saturated sigmoids
    gu[M // 3, :I] = -80.0
    dh[M // 4] = 0.0
    return gu, dh


@pytest.mark.parametrize("M,I,dual", [(1, 128, False), (5, 256, False), (77, 384, False), (300, 2816, False), (1000, 128, False),
                                      (128, 128, True), (384, 1024, True), (4096, 2816, True), (4096, 2816, False)])
def test_forward(fp8lib, M, I, dual):
    gu, _ = make(M, I, 3 * M + I)
    q, s, qT, sT, qgu, sgu = fp8lib.silu_mul_quant_ckpt(gu, dual=dual)
    want = (*fp8lib.silu_mul_quant(gu, dual=dual), *fp8lib.quantize_1x128(gu))
    for a, b in zip((q, s, qT, sT, qgu, sgu), want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert fp8lib.check_status() == _abi.FP8RL_OK


def test_forward_tiny_scales(fp8lib):
    """Groups whose scale is too small for the division-free encode."""
    gu, _ = make(128, 256, 5)
    gu[3] = gu[3].float().mul(2.0 ** -80).to(torch.bfloat16)
    gu[:, 128:256] = gu[:, 128:256].float().mul(2.0 ** -75).to(torch.bfloat16)
    got = fp8lib.silu_mul_quant_ckpt(gu)
    for a, b in zip(got, (*fp8lib.silu_mul_quant(gu), *fp8lib.quantize_1x128(gu))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,I,dual", [(1, 128, False), (77, 384, False), (300, 2816, False), (128, 128, True), (384, 1024, True), (4096, 2816, True)])
def test_backward_of_exact_checkpoint(fp8lib, M, I, dual):
    """Power-of-two scales: decode(code) * scale is a BF16 number, so the bits are those of the
    BF16 operator on it."""
    gen = torch.Generator("cuda").manual_seed(M + I)
    q = torch.randint(0, 256, (M, 2 * I), generator=gen, device="cuda", dtype=torch.uint8)
    q[(q & 0x7F) == 0x7F] = 0          # no NaN codes
    s = torch.exp2(torch.randint(-12, -5, (2 * I // 128, M), generator=gen, device="cuda").float())
    gu = ref.decode((q, s)).to(torch.bfloat16)
    assert torch.equal(gu.double(), ref.decode((q, s)))
    dh = synth.normal_bf16((M, I), 1e-3, 7, "cuda")
    got = fp8lib.silu_mul_bwd_quant_ckpt(q, s, dh, dual=dual)
    want = fp8lib.silu_mul_bwd_quant(gu, dh, dual=dual)
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert fp8lib.check_status() == _abi.FP8RL_OK


def gradient(gu, dh):
    I = dh.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    sg = torch.sigmoid(g)
    d = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1)
    mag = torch.cat([(dh * u).abs() * sg * (1 + (g * (1 - sg)).abs()), (dh * g).abs() * sg], 1)
    return d, mag


def check_codes(q, s, d, mag):
    M, C = q.shape
    err = mag * 2.0 ** -16 + 2.0 ** -134
    group = lambda x: x.view(M, C // 128, 128)  # noqa: E731
    amax = group(d.abs()).amax(2)
    slack = group(err).amax(2) + ref.BF16_HALF * amax
    got = 448.0 * s.double().t()
    assert bool(((got - amax).abs() <= slack + 2.0 ** -22 * amax).all())
    bound = (2.0 ** -4 + ref.BF16_HALF) * d.abs() + 2 * err + (2.0 ** -10 * s.double().t()).unsqueeze(2).expand(M, C // 128, 128).reshape(M, C)
    bad = (ref.decode((q, s)) - d).abs() > bound * (1 + 2.0 ** -4)
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("M,I,dual", [(1, 128, False), (3, 256, False), (77, 384, False), (300, 2816, False), (128, 128, True), (384, 1024, True)])
def test_backward(fp8lib, M, I, dual):
    gu, dh = make(M, I, 5 * M + I)
    *_, qgu, sgu = fp8lib.silu_mul_quant_ckpt(gu, dual=False)
    q, s, qT, sT = fp8lib.silu_mul_bwd_quant_ckpt(qgu, sgu, dh, dual=dual)
    d, mag = gradient(ref.decode((qgu, sgu)), dh.double())
    check_codes(q, s, d, mag)
    if dual:
        check_codes(qT, sT, d.t().contiguous(), mag.t().contiguous())
    again = fp8lib.silu_mul_bwd_quant_ckpt(qgu, sgu, dh, dual=dual)
    for a, b in zip((q, s, qT, sT), again):
        assert a is None or torch.equal(a, b)
    assert fp8lib.check_status() == _abi.FP8RL_OK


def test_backward_formula_against_differences():
    gen = torch.Generator("cuda").manual_seed(1)
    gu = torch.randn((4, 64), generator=gen, device="cuda", dtype=torch.float64)
    dh = torch.randn((4, 32), generator=gen, device="cuda", dtype=torch.float64)
    v = torch.randn((4, 64), generator=gen, device="cuda", dtype=torch.float64)
    f = lambda x: float((torch.nn.functional.silu(x[:, :32]) * x[:, 32:] * dh).sum())  # noqa: E731
    diff = (f(gu + 1e-5 * v) - f(gu - 1e-5 * v)) / 2e-5
    assert abs(diff - float((gradient(gu, dh)[0] * v).sum())) <= 1e-7 * (1 + abs(diff))


def test_on_another_stream_and_captured(fp8lib):
    M, I = 256, 384
    gu, dh = make(M, I, 2)

    def step():
        f = fp8lib.silu_mul_quant_ckpt(gu)
        return (*f, *fp8lib.silu_mul_bwd_quant_ckpt(f[4], f[5], dh))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, cap):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_no_rows(fp8lib):
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q, s, qT, sT, qgu, sgu = fp8lib.silu_mul_quant_ckpt(e)
    assert q.shape == (0, 128) and qT.shape == (128, 0) and qgu.shape == (0, 256)
    d = fp8lib.silu_mul_bwd_quant_ckpt(qgu, sgu, torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"))
    assert d[0].shape == (0, 256)
