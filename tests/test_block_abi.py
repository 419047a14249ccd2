"""Host-side argument checks of the block operators: every refusal answers without a GPU and
launches nothing (the pointers are never dereferenced)."""
import ctypes

import pytest

FAKE, ODD = 0x10000, 0x10004


@pytest.fixture(scope="module")
def abi():
    from block_scaled_fp8_x1_gb300 import build_library
    from block_scaled_fp8_x1_gb300 import _abi
    build_library()
    return _abi


def norm_args(abi, **kw):
    base = dict(h=FAKE, ldh=256, y=FAKE, ldy=256, pre_gamma=FAKE, alpha=1.0, eps=1e-5, h_out=FAKE + 4096, z=FAKE,
                r_pre=FAKE)
    return abi.ResidualNormArgs(**{**base, **kw})


@pytest.mark.parametrize("kw,M,K,status", [
    ({}, -1, 256, "INVALID_ARG"), ({}, 4, 0, "INVALID_ARG"), ({}, 4, 200, "SHAPE"), ({}, 4, 8320, "SHAPE"),
    (dict(eps=-1.0), 4, 256, "INVALID_ARG"), (dict(eps=float("nan")), 4, 256, "INVALID_ARG"),
    (dict(alpha=float("inf")), 4, 256, "INVALID_ARG"), (dict(alpha=float("nan")), 4, 256, "INVALID_ARG"),
    (dict(h=None), 4, 256, "INVALID_ARG"), (dict(y=None), 4, 256, "INVALID_ARG"),
    (dict(pre_gamma=None), 4, 256, "INVALID_ARG"), (dict(h_out=None), 4, 256, "INVALID_ARG"),
    (dict(r_pre=None), 4, 256, "INVALID_ARG"), (dict(post_gamma=FAKE), 4, 256, "INVALID_ARG"),
    (dict(z=None), 4, 256, "INVALID_ARG"), (dict(q=FAKE), 4, 256, "INVALID_ARG"),
    (dict(sT=FAKE), 128, 256, "INVALID_ARG"), (dict(qh=FAKE), 4, 256, "INVALID_ARG"),
    (dict(sy=FAKE), 4, 256, "INVALID_ARG"), (dict(qT=FAKE, sT=FAKE), 100, 256, "SHAPE"),
    (dict(ldh=128), 4, 256, "INVALID_ARG"), (dict(ldy=128), 4, 256, "INVALID_ARG"),
    (dict(ldy=260), 4, 256, "ALIGN"), (dict(h=ODD), 4, 256, "ALIGN"), (dict(z=ODD), 4, 256, "ALIGN"),
    (dict(gate=ODD), 4, 256, "ALIGN"), (dict(q=FAKE, s=ODD), 4, 256, "ALIGN"), (dict(r_pre=ODD), 4, 256, "ALIGN"),
    (dict(h_out=FAKE, ldh=264), 4, 256, "INVALID_ARG"),
    (dict(h=None, y=None, z=None), 0, 256, "OK"),
])
def test_residual_norm_refusals(abi, kw, M, K, status):
    want = getattr(abi, "FP8RL_OK" if status == "OK" else f"FP8RL_ERR_{status}")
    assert abi.lib().fp8rl_residual_norm(ctypes.byref(norm_args(abi, **kw)), M, K, None) == want


def bwd_args(abi, **kw):
    base = dict(dz=FAKE, lddz=256, dh=FAKE, lddh=256, h=FAKE, ldh=256, y=FAKE, ldy=256, pre_gamma=FAKE, alpha=1.0,
                r_pre=FAKE, dh_out=FAKE, dy=FAKE, dpre=FAKE)
    return abi.ResidualNormBwdArgs(**{**base, **kw})


GATED = dict(gate=FAKE, dgate=FAKE)


@pytest.mark.parametrize("kw,M,K,status", [
    ({}, -1, 256, "INVALID_ARG"), ({}, 4, 200, "SHAPE"), ({}, 4, 8320, "SHAPE"),
    (dict(alpha=float("nan")), 4, 256, "INVALID_ARG"), (dict(dz=None), 4, 256, "INVALID_ARG"),
    (dict(h=None), 4, 256, "INVALID_ARG"), (dict(r_pre=None), 4, 256, "INVALID_ARG"),
    (dict(dpre=None), 4, 256, "INVALID_ARG"), (dict(dy=None), 4, 256, "INVALID_ARG"),
    (dict(gate=FAKE), 4, 256, "INVALID_ARG"), (dict(post_gamma=FAKE, r_post=FAKE), 4, 256, "INVALID_ARG"),
    (dict(post_gamma=FAKE, dpost=FAKE), 4, 256, "INVALID_ARG"), (dict(qh=FAKE), 4, 256, "INVALID_ARG"),
    (dict(y=None, **GATED), 4, 256, "INVALID_ARG"), (dict(qh=FAKE, sh=FAKE, **GATED), 4, 256, "INVALID_ARG"),
    (dict(qy=FAKE, sy=FAKE, **GATED), 4, 256, "INVALID_ARG"), (dict(lddz=128), 4, 256, "INVALID_ARG"),
    (dict(lddh=252), 4, 256, "INVALID_ARG"), (dict(ldh=260), 4, 256, "ALIGN"), (dict(dz=ODD), 4, 256, "ALIGN"),
    (dict(dpre=ODD), 4, 256, "ALIGN"), (dict(qh=FAKE, sh=ODD), 4, 256, "ALIGN"),
])
def test_residual_norm_bwd_refusals(abi, kw, M, K, status):
    want = getattr(abi, f"FP8RL_ERR_{status}")
    L = abi.lib()
    assert L.fp8rl_residual_norm_bwd(ctypes.byref(bwd_args(abi, **kw)), M, K, FAKE, 1 << 30, None) == want


def test_residual_norm_bwd_workspace(abi):
    f = abi.lib().fp8rl_residual_norm_bwd_workspace_bytes
    assert f(0, 256) == 0 and f(4, 200) == 0 and f(4, 8320) == 0
    assert f(1, 256) == 2 * 256 * 4                    # one row, one block
    assert f(1 << 20, 5120) <= 160 * 2 * 5120 * 4      # one block per SM at this width


@pytest.mark.parametrize("M,I,ptr,status", [
    (-1, 256, {}, "INVALID_ARG"), (4, 0, {}, "INVALID_ARG"), (4, 200, {}, "SHAPE"), (100, 256, dict(qT=FAKE, sT=FAKE), "SHAPE"),
    (4, 256, dict(qT=FAKE), "INVALID_ARG"), (4, 256, dict(src=None), "INVALID_ARG"), (4, 256, dict(ck=None), "INVALID_ARG"),
    (4, 256, dict(sck=None), "INVALID_ARG"), (4, 256, dict(q=None), "INVALID_ARG"), (4, 256, dict(src=ODD), "ALIGN"),
    (4, 256, dict(ck=ODD), "ALIGN"), (4, 256, dict(sck=ODD), "ALIGN"), (128, 256, dict(qT=ODD, sT=FAKE), "ALIGN"),
    (0, 256, dict(src=None, ck=None, sck=None, q=None), "OK"),
])
def test_silu_checkpoint_refusals(abi, M, I, ptr, status):
    p = {**dict(src=FAKE, q=FAKE, s=FAKE, qT=None, sT=None, ck=FAKE, sck=FAKE), **ptr}
    want = getattr(abi, "FP8RL_OK" if status == "OK" else f"FP8RL_ERR_{status}")
    L = abi.lib()
    assert L.fp8rl_silu_mul_quant_ckpt(p["src"], M, I, p["q"], p["s"], p["qT"], p["sT"], p["ck"], p["sck"], None) == want
    assert L.fp8rl_silu_mul_bwd_quant_ckpt(p["ck"], p["sck"], p["src"], M, I, p["q"], p["s"], p["qT"], p["sT"], None) == want


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "INVALID_ARG"), (dict(N=-1), "INVALID_ARG"), (dict(K=0), "INVALID_ARG"), (dict(ldx=128), "INVALID_ARG"),
    (dict(ldy=64), "INVALID_ARG"), (dict(splits=-1), "INVALID_ARG"), (dict(splits=9), "INVALID_ARG"), (dict(M=17), "SHAPE"),
    (dict(K=384, ldx=384), "SHAPE"), (dict(N=200, ldy=200), "SHAPE"), (dict(x=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"),
    (dict(sf=None), "INVALID_ARG"), (dict(g=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(x=ODD), "ALIGN"),
    (dict(q=ODD), "ALIGN"), (dict(sf=ODD), "ALIGN"), (dict(g=ODD), "ALIGN"), (dict(y=ODD), "ALIGN"), (dict(ldx=260), "ALIGN"),
    (dict(ldy=132), "ALIGN"), (dict(M=0, x=None, y=None), "OK"), (dict(N=0, q=None, ldy=0), "OK"),
])
def test_matvec_nvfp4_refusals(abi, kw, status):
    a = {**dict(x=FAKE, M=4, K=256, ldx=256, q=FAKE, sf=FAKE, g=FAKE, N=128, y=FAKE, ldy=128, splits=0), **kw}
    want = getattr(abi, "FP8RL_OK" if status == "OK" else f"FP8RL_ERR_{status}")
    assert abi.lib().fp8rl_matvec_nvfp4(a["x"], a["M"], a["K"], a["ldx"], a["q"], a["sf"], a["g"], a["N"], a["y"], a["ldy"],
                                        a["splits"], None) == want


def test_binding_refuses_what_is_not_on_a_gpu_or_has_another_type():
    """The binding's own checks answer before any CUDA call."""
    import torch
    from block_scaled_fp8_x1_gb300 import ops
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for call in (lambda x: ops.residual_norm(x, x, b(256), 1e-5), lambda x: ops.residual_norm_bwd(x, x, x, x, b(256), b(4)),
                 lambda x: ops.silu_mul_quant_ckpt(x), lambda x: ops.matvec_nvfp4(x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call(b(4, 256))
        with pytest.raises(TypeError):
            call(torch.zeros((4, 256)))
        with pytest.raises(ValueError, match="matrix"):
            call(b(256))
    with pytest.raises(TypeError):
        ops.silu_mul_bwd_quant_ckpt(b(4, 256), b(2, 4), b(4, 128))
