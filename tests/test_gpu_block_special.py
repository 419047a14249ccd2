"""Infinities, NaN, sums outside FP32 and eps = 0 in the norms either side of a block and in the SiLU
operators with an 8-bit checkpoint.

The codes of a group of 128 that holds an infinity or a NaN are unspecified; its scale is not finite, and
the other groups are those of the stand-alone operators bit for bit."""
import pytest
import torch

import test_gpu_residual_norm as base
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def check_codes(got, want):
    """(codes [M,C], scales [C/128,M]) equal in every group whose scale is finite."""
    (q, s), (wq, ws) = got, want
    fine = torch.isfinite(ws)
    assert torch.equal(torch.isfinite(s), fine) and torch.equal(s[fine], ws[fine])
    M, C = q.shape
    g, wg = (x.view(M, C // 128, 128).transpose(0, 1) for x in (q, wq))
    assert torch.equal(g[fine], wg[fine])
    return fine


def finite_groups(x):
    return torch.isfinite(x).view(x.shape[0], -1, 128).all(2).t()


@pytest.mark.parametrize("K", [256, 3584, 8192])
@pytest.mark.parametrize("post", [False, True])
def test_norm_rows_with_special_values(fp8lib, K, post):
    M = 12
    h, y, pre, post_g, gate = base.inputs(M, K, post, True)
    kw = dict(post_gamma=post_g, gate=gate, checkpoint=True)
    want = fp8lib.residual_norm(h, y, pre, base.EPS, emit="fp8", **kw)
    want_z = fp8lib.residual_norm(h, y, pre, base.EPS, emit="bf16", **kw).z
    h[1, 5] = INF
    h[3, K - 1] = NAN
    h[5] = 3e25                        # squares past FP32's range: r = 0
    y[7, 9] = NAN
    y[9, 11] = -INF
    y[10] = 1e30
    r = fp8lib.residual_norm(h, y, pre, base.EPS, emit="fp8", **kw)
    z = fp8lib.residual_norm(h, y, pre, base.EPS, emit="bf16", **kw)
    for m in (0, 2, 4, 6, 8, 11):      # the other rows
        for a, b in zip((r.h, r.r_pre, r.q, z.z, r.h_ckpt[0], r.y_ckpt[0]), (want.h, want.r_pre, want.q, want_z, want.h_ckpt[0], want.y_ckpt[0])):
            assert torch.equal(a[m], b[m])
        for a, b in ((r.s, want.s), (r.h_ckpt[1], want.h_ckpt[1]), (r.y_ckpt[1], want.y_ckpt[1])):
            assert torch.equal(a[:, m], b[:, m])
    # an infinite sum of squares has r = 0; what was finite becomes 0, the infinity itself NaN
    assert float(r.r_pre[1]) == 0.0 and float(r.r_pre[5]) == 0.0
    rest = torch.arange(K, device="cuda") != 5
    assert bool((z.z[1][rest] == 0).all()) and bool(torch.isnan(z.z[1, 5]))
    assert bool((z.z[5] == 0).all()) and bool(torch.isfinite(r.h[5]).all())
    assert bool(torch.isnan(r.r_pre[3])) and bool(torch.isnan(z.z[3]).all())
    assert int(torch.isnan(r.h[3]).sum()) == 1
    if post:
        assert float(r.r_post[9]) == 0.0 and float(r.r_post[10]) == 0.0 and bool(torch.isnan(r.r_post[7]))
        assert torch.equal(r.h[10], h[10])                       # y r = 0
        rest = torch.arange(K, device="cuda") != 11
        assert torch.equal(r.h[9][rest], h[9][rest]) and bool(torch.isnan(r.h[9, 11]))
    else:
        assert int(torch.isnan(r.h[7]).sum()) == 1 and float(r.r_pre[9]) == 0.0 and float(r.r_pre[10]) == 0.0
    for got, x in (((r.q, r.s), z.z), (r.h_ckpt, r.h), (r.y_ckpt, y)):
        assert torch.equal(check_codes(got, fp8lib.quantize_1x128(x)), finite_groups(x))
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("post", [False, True])
def test_norm_without_eps(fp8lib, post):
    """eps = 0: the formula as it is, 1/sqrt(0) in a row of zeros."""
    M, K = 9, 640
    h, y, pre, post_g, _ = base.inputs(M, K, post, False)
    h[2] = y[2] = 0.0
    r = fp8lib.residual_norm(h, y, pre, 0.0, post_gamma=post_g, emit="bf16")
    rest = [0, 1, 3, 4, 5, 6, 7, 8]
    exact = r.h[rest].double().square().mean(1).rsqrt()
    # r within the bound of the other sizes, z one BF16 rounding more
    assert bool(((r.r_pre[rest].double() - exact).abs() <= 2.0 ** -18 * exact).all())
    z = r.h[rest].double() * exact[:, None] * pre.double()
    assert bool(((r.z[rest].double() - z).abs() <= (2.0 ** -8 + 2.0 ** -17) * z.abs()).all())
    if post:
        assert float(r.r_post[2]) == INF and bool(torch.isnan(r.h[2]).all())
    else:
        assert float(r.r_pre[2]) == INF and bool((r.h[2] == 0).all())
    assert bool(torch.isnan(r.z[2]).all())


def test_norm_backward_keeps_a_nan_in_its_row(fp8lib):
    M, K = 300, 640
    h, y, pre, post, gate = base.inputs(M, K, True, True)
    f = fp8lib.residual_norm(h, y, pre, base.EPS, post_gamma=post, gate=gate, checkpoint=True)
    dz = synth.normal_bf16((M, K), 1e-3, 21, "cuda")
    for hs, ys in ((f.h, y), (f.h_ckpt, f.y_ckpt)):
        run = lambda d: fp8lib.residual_norm_bwd(d, dz, hs, ys, pre, f.r_pre, post_gamma=post, r_post=f.r_post, gate=gate)  # noqa: E731
        want, bad = run(dz), dz.clone()
        bad[7, 3] = NAN
        got = run(bad)
        rest = torch.arange(M, device="cuda") != 7
        assert torch.equal(got.dh[rest], want.dh[rest]) and torch.equal(got.dy[rest], want.dy[rest])
        assert bool(torch.isnan(got.dh[7]).all()) and bool(torch.isnan(got.dy[7]).all())


@pytest.mark.parametrize("M,I,dual", [(5, 128, False), (128, 256, True), (77, 384, False)])
def test_silu_with_special_values(fp8lib, M, I, dual):
    gu = synth.normal_bf16((M, 2 * I), 1.5, 3, "cuda")
    gu[0, 3], gu[0, I + 7] = INF, -INF
    gu[1, 5], gu[1, 9] = -INF, NAN
    gu[2, I + 1] = NAN
    gu[3, :64] = 3e38
    gu[4, :64] = -3e38
    q, s, qT, sT, qgu, sgu = fp8lib.silu_mul_quant_ckpt(gu, dual=dual)
    want = fp8lib.silu_mul_quant(gu, dual=dual)
    assert not bool(check_codes((q, s), want[:2])[0, 0])
    if dual:
        check_codes((qT, sT), want[2:])
    assert torch.equal(check_codes((qgu, sgu), fp8lib.quantize_1x128(gu)), finite_groups(gu))
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("M,I,dual", [(5, 128, False), (128, 256, True), (77, 384, False)])
def test_silu_backward_with_special_values(fp8lib, M, I, dual):
    """Codes with power-of-two scales decode to BF16 numbers: the codes of the BF16 operator."""
    gen = torch.Generator("cuda").manual_seed(M + I)
    q = torch.randint(0, 256, (M, 2 * I), generator=gen, device="cuda", dtype=torch.uint8)
    q[(q & 0x7F) == 0x7F] = 0
    q[1, 5] = 0x7F                     # a NaN code
    s = torch.exp2(torch.randint(-12, -5, (2 * I // 128, M), generator=gen, device="cuda").float())
    s[0, 2], s[-1, 3] = 2.0 ** 119, NAN
    group = q.view(torch.float8_e4m3fn).float().view(M, 2 * I // 128, 128)
    gu = (group * s.t().unsqueeze(2)).view(M, 2 * I).to(torch.bfloat16)
    dh = synth.normal_bf16((M, I), 1e-3, 7, "cuda")
    dh[0, 3], dh[4, 4] = INF, NAN
    got = fp8lib.silu_mul_bwd_quant_ckpt(q, s, dh, dual=dual)
    want = fp8lib.silu_mul_bwd_quant(gu, dh, dual=dual)
    assert not bool(check_codes(got[:2], want[:2]).all())
    if dual:
        check_codes(got[2:], want[2:])
    assert fp8lib.check_status() == _abi.FP8RL_OK
