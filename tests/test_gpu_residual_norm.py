"""The norms before and after a block with its gate and residual scale, on the GPU, against the
64-bit definition.

Bounds count roundings (bf16: half a step is 2^-8 of the value, fp32: 2^-24).  A row's sum of
squares is chained over at most 8 + 5 + 32 additions and its root halves the error: r is within
2^-18.  h' has one bf16 rounding and at most 16 fp32 roundings (2^-20) of its terms' magnitudes,
beside r's error in the branch.  The gradients' row sums chain at most 16 + 5 + 32 additions and
their elements fewer than 32 more roundings: 2^-17 of the terms' magnitudes, twice that through
the second norm; the column sums add at most 130 rows in one block and 160 / 8 + 8 partial sums:
2^-15 of the terms' magnitudes, which covers the elements' own error.
"""
import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu
EPS = 1e-5


def gains(K, seed):
    return (1.0 + 0.1 * torch.randn(K, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")).to(torch.bfloat16)


def inputs(M, K, post, gated, seed=0):
    out = max(1, K // 1000)
    h = synth.normal_bf16((M, K), 1.0, 11 + seed, "cuda", outlier_channels=out, outlier_scale=30.0)
    y = synth.normal_bf16((M, K), 0.7, 12 + seed, "cuda", outlier_channels=out, outlier_scale=30.0)
    return h, y, gains(K, 13), gains(K, 14) if post else None, gains(K, 15) if gated else None


def d64(t):
    return None if t is None else t.double()


def check(name, got, value, bound):
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {err.numel()} outside, worst {float((err - bound).max()):.3e}"


def check_forward(r, h, y, pre, post, gate, alpha):
    want = ref.residual_norm(d64(h), d64(y), d64(pre), EPS, d64(post), d64(gate), alpha)
    t = (want[0] - h.double()).abs()
    check("h'", r.h, want[0], ref.BF16_HALF * want[0].abs() + 2.0 ** -17 * t + 2.0 ** -20 * h.double().abs())
    rp = ref.rstd(r.h.double(), EPS)
    check("r_pre", r.r_pre, rp, 2.0 ** -18 * rp)
    if post is not None:
        check("r_post", r.r_post, want[3], 2.0 ** -18 * want[3])
    z = r.h.double() * rp[:, None] * pre.double()
    if r.z is not None:
        check("z", r.z, z, (ref.BF16_HALF + 2.0 ** -17) * z.abs())


SHAPES = [(1, 128), (1, 3584), (1, 8192), (2, 640), (3, 1152), (77, 5120), (300, 640), (613, 4096), (1000, 256), (129, 8192)]


@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(fp8lib, M, K, post, gated):
    h, y, pre, post_g, gate = inputs(M, K, post, gated)
    y[0] = 0.0                                     # a zero row: r = 1/sqrt(eps)
    if M > 1:
        h[1] = 0.0
        y[1] = 0.0                                 # and one whose h' is zero too
    r = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post_g, gate=gate, alpha=0.5, emit="bf16", checkpoint=True)
    check_forward(r, h, y, pre, post_g, gate, 0.5)
    # the quantized forms are the quantizers' of the same tensors, bit for bit
    f = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post_g, gate=gate, alpha=0.5, emit="fp8")
    assert torch.equal(f.h, r.h) and torch.equal(f.r_pre, r.r_pre)
    for got, x in (((f.q, f.s), r.z), (r.h_ckpt, r.h), (r.y_ckpt, y)):
        q, s = fp8lib.quantize_1x128(x)
        assert torch.equal(got[0], q) and torch.equal(got[1], s)
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("M,K", [(128, 128), (384, 640), (1024, 5120), (256, 8192)])
def test_forward_dual(fp8lib, M, K):
    h, y, pre, post, gate = inputs(M, K, True, True)
    r = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="dual")
    z = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="bf16").z
    q, s, qT, sT = fp8lib.quantize_1x128(z, dual=True)
    for a, b in ((r.q, q), (r.s, s), (r.qT, qT), (r.sT, sT)):
        assert torch.equal(a, b)
    assert fp8lib.check_status() == _abi.FP8RL_OK


def test_a_row_alone_has_the_bits_it_has_in_a_batch(fp8lib):
    M, K = 2000, 3584
    h, y, pre, post, gate = inputs(M, K, True, True)
    all_ = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="bf16")
    for m in (0, 5, 1999):
        one = fp8lib.residual_norm(h[m:m + 1], y[m:m + 1], pre, EPS, post_gamma=post, gate=gate, emit="bf16")
        for f in ("h", "z", "r_pre", "r_post"):
            assert torch.equal(getattr(one, f)[0], getattr(all_, f)[m]), (m, f)


def test_strides_inplace_and_another_stream(fp8lib):
    M, K = 77, 640
    h, y, pre, post, gate = inputs(M, K, True, True)
    want = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="bf16")
    wide_h = torch.full((M, K + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_y = torch.full((2 * M, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_h[:, 64:64 + K] = h
    wide_y[::2, :K] = y
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fp8lib.residual_norm(wide_h[:, 64:64 + K], wide_y[::2, :K], pre, EPS, post_gamma=post, gate=gate, emit="bf16")
        mine = h.clone()
        inpl = fp8lib.residual_norm(mine, y, pre, EPS, post_gamma=post, gate=gate, emit="bf16", inplace=True)
    side.synchronize()
    assert inpl.h.data_ptr() == mine.data_ptr()
    for r in (got, inpl):
        for f in ("h", "z", "r_pre", "r_post"):
            assert torch.equal(getattr(r, f), getattr(want, f)), f


def test_rows_far_apart(fp8lib):
    """Row offsets past 2^31 elements."""
    K, ld = 256, 1 << 30
    h, y, pre, post, gate = inputs(4, K, True, True)
    base = torch.empty(3 * ld + K, dtype=torch.bfloat16, device="cuda")
    far = base.as_strided((4, K), (ld, 1))
    far.copy_(y)
    want = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="bf16")
    got = fp8lib.residual_norm(h, far, pre, EPS, post_gamma=post, gate=gate, emit="bf16")
    assert torch.equal(got.h, want.h) and torch.equal(got.z, want.z)


# ---------------------------------------------------------------- backward

@pytest.mark.parametrize("saved", ["bf16", "fp8"])
@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 8192), (2, 640), (77, 5120), (300, 640), (613, 4096), (1000, 256), (400, 8192), (3000, 1152), (37, 5248)])
def test_backward(fp8lib, M, K, post, gated, saved):
    alpha = 0.5
    h, y, pre, post_g, gate = inputs(M, K, post, gated, seed=5)
    if M > 1:
        h[1] = 0.0
        y[1] = 0.0
    f = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post_g, gate=gate, alpha=alpha, emit="fp8", checkpoint=True)
    dz = synth.normal_bf16((M, K), 1e-3, 21, "cuda")
    dh = synth.normal_bf16((M, K), 1e-3, 22, "cuda")
    hs, ys = (f.h, y) if saved == "bf16" else (f.h_ckpt, f.y_ckpt)
    kw = dict(post_gamma=post_g, r_post=f.r_post, gate=gate, alpha=alpha)
    g = fp8lib.residual_norm_bwd(dz, dh, hs, ys, pre, f.r_pre, **kw)
    want = ref.residual_norm_bwd(d64(dz), d64(dh), ref.decode(hs), ref.decode(ys), d64(pre), d64(f.r_pre),
                                 d64(post_g), d64(f.r_post), d64(gate), alpha)
    got = {"dh": g.dh, "dy": g.dy, "dpre": g.dpre}
    if post:
        got["dpost"] = g.dpost
    if gated:
        got["dgate"] = g.dgate
    assert set(got) == set(want) and (g.dpost is None) == (not post) and (g.dgate is None) == (not gated)
    for k, (v, mag) in want.items():
        if k in ("dh", "dy"):
            check(k, got[k], v, ref.BF16_HALF * v.abs() + 2.0 ** (-17 if k == "dh" else -16) * mag)
        else:
            check(k, got[k], v, 2.0 ** -15 * mag)
    # the sums run in a fixed order
    again = fp8lib.residual_norm_bwd(dz, dh, hs, ys, pre, f.r_pre, **kw)
    for a, b in zip(g, again):
        assert a is None or torch.equal(a, b)
    # no gradient from above is a gradient of zero
    none = fp8lib.residual_norm_bwd(dz, None, hs, ys, pre, f.r_pre, **kw)
    zero = fp8lib.residual_norm_bwd(dz, torch.zeros_like(dh), hs, ys, pre, f.r_pre, **kw)
    for a, b in zip(none, zero):
        assert a is None or torch.equal(a, b)


def test_backward_against_differences(fp8lib):
    """The kernel's gradients along random directions against central differences of the 64-bit
    forward.  Each product sums elements with a bf16 rounding of the gradient and of the saved h'
    (2^-8 of the element's terms each), independent of each other: within 8 times
    2^-7 sqrt(sum (mag d)^2)."""
    M, K, alpha, step = 64, 640, 0.5, 1e-4
    h, y, pre, post, gate = inputs(M, K, True, True, seed=9)
    dz = synth.normal_bf16((M, K), 1.0, 31, "cuda")
    dh = synth.normal_bf16((M, K), 1.0, 32, "cuda")
    v = {"h": d64(h), "y": d64(y), "pre": d64(pre), "post": d64(post), "gate": d64(gate)}

    def forward(v):
        return ref.residual_norm(v["h"], v["y"], v["pre"], EPS, v["post"], v["gate"], alpha)

    h2, _, r, rp = forward(v)
    # the rounding of h' is passed straight through
    g = fp8lib.residual_norm_bwd(dz, dh, h2.to(torch.bfloat16), y, pre, r.float(), post_gamma=post, r_post=rp.float(),
                                 gate=gate, alpha=alpha)
    exact = ref.residual_norm_bwd(d64(dz), d64(dh), h2, d64(y), d64(pre), r, d64(post), rp, d64(gate), alpha)
    gen = torch.Generator("cuda").manual_seed(4)
    for name, got, full in (("h", g.dh, "dh"), ("y", g.dy, "dy"), ("pre", g.dpre, "dpre"), ("post", g.dpost, "dpost"),
                            ("gate", g.dgate, "dgate")):
        d = torch.randn(v[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        loss = []
        for sgn in (1, -1):
            a, z, _, _ = forward({**v, name: v[name] + sgn * step * d})
            loss.append(float((z * d64(dz)).sum() + (a * d64(dh)).sum()))
        diff = (loss[0] - loss[1]) / (2 * step)
        tol = 8 * 2 * ref.BF16_HALF * float((exact[full][1] * d).square().sum().sqrt()) + 1e-5 * abs(diff)
        assert abs(float((got.double() * d).sum()) - diff) <= tol, name


def test_backward_strides_and_stream(fp8lib):
    M, K = 301, 1152
    h, y, pre, post, gate = inputs(M, K, True, True)
    f = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="fp8")
    dz = synth.normal_bf16((M, K), 1e-3, 21, "cuda")
    dh = synth.normal_bf16((M, K), 1e-3, 22, "cuda")
    kw = dict(post_gamma=post, r_post=f.r_post, gate=gate)
    want = fp8lib.residual_norm_bwd(dz, dh, f.h, y, pre, f.r_pre, **kw)
    wide = [torch.full((M, K + 16), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    views = []
    for w, t in zip(wide, (dz, dh, f.h, y)):
        w[:, 8:8 + K] = t
        views.append(w[:, 8:8 + K])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fp8lib.residual_norm_bwd(*views, pre, f.r_pre, **kw)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_into_a_graph(fp8lib):
    M, K = 256, 1152
    h, y, pre, post, gate = inputs(M, K, True, True)
    dz = synth.normal_bf16((M, K), 1e-3, 21, "cuda")

    def step():
        f = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, emit="dual", checkpoint=True)
        return f, fp8lib.residual_norm_bwd(dz, dz, f.h_ckpt, f.y_ckpt, pre, f.r_pre, post_gamma=post,
                                           r_post=f.r_post, gate=gate)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, g = step()
    y.copy_(synth.normal_bf16((M, K), 0.7, 99, "cuda"))
    graph.replay()
    torch.cuda.synchronize()
    f2, g2 = step()
    for a, b in zip((f.h, f.q, f.qT, *g), (f2.h, f2.q, f2.qT, *g2)):
        assert torch.equal(a, b)


def test_no_rows(fp8lib):
    K = 256
    _, _, pre, post, gate = inputs(1, K, True, True)
    e = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    r = fp8lib.residual_norm(e, e, pre, EPS, post_gamma=post, gate=gate, emit="dual", checkpoint=True)
    assert r.h.shape == (0, K) and r.q.shape == (0, K) and r.qT.shape == (K, 0)
    g = fp8lib.residual_norm_bwd(e, e, e, e, pre, r.r_pre, post_gamma=post, r_post=r.r_post, gate=gate)
    assert g.dh.shape == (0, K)
    for v in (g.dpre, g.dpost, g.dgate):
        assert float(v.abs().max()) == 0.0


def test_refusals(fp8lib):
    M, K = 4, 256
    h, y, pre, post, gate = inputs(M, K, True, True)
    with pytest.raises(ValueError, match="y: expected shape"):
        fp8lib.residual_norm(h, y[:3], pre, EPS)
    with pytest.raises(ValueError, match="contiguous"):
        fp8lib.residual_norm(h.t().contiguous().t(), y, pre, EPS)
    with pytest.raises(ValueError, match="pre_gamma"):
        fp8lib.residual_norm(h, y, pre[:128], EPS)
    with pytest.raises(ValueError, match="pre_gamma"):
        fp8lib.residual_norm(h, y, None, EPS)
    with pytest.raises(ValueError, match="emit"):
        fp8lib.residual_norm(h, y, pre, EPS, emit="int8")
    with pytest.raises(ValueError, match="on cpu|CUDA"):
        fp8lib.residual_norm(h, y.cpu(), pre, EPS)
    with pytest.raises(_abi.Fp8rlError) as e:
        fp8lib.residual_norm(h, y, pre, EPS, emit="dual")          # M % 128
    assert e.value.status == _abi.FP8RL_ERR_SHAPE
    with pytest.raises(_abi.Fp8rlError) as e:
        fp8lib.residual_norm(h[:, :200], y[:, :200], pre[:200], EPS)
    assert e.value.status == _abi.FP8RL_ERR_SHAPE
    f = fp8lib.residual_norm(h, y, pre, EPS, post_gamma=post, gate=gate, checkpoint=True)
    dz = torch.zeros_like(h)
    with pytest.raises(ValueError, match="r_post"):
        fp8lib.residual_norm_bwd(dz, dz, f.h, y, pre, f.r_pre, post_gamma=post)
    with pytest.raises(ValueError, match="y: needed"):
        fp8lib.residual_norm_bwd(dz, dz, f.h, None, pre, f.r_pre, gate=gate)
    with pytest.raises(ValueError, match="both"):
        fp8lib.residual_norm_bwd(dz, dz, f.h_ckpt, y, pre, f.r_pre, gate=gate)
    with pytest.raises(ValueError, match="h scales"):
        fp8lib.residual_norm_bwd(dz, dz, (f.h_ckpt[0], f.h_ckpt[1].t()), None, pre, f.r_pre)
