"""Every set of outputs that fp8rl_residual_norm accepts, through the C call: each output bit for bit what
the stand-alone operators make of the same tensors, and nothing written beside it."""
import ctypes
import itertools

import pytest
import torch

import test_gpu_residual_norm as base
from block_scaled_fp8_x1_gb300 import _abi

pytestmark = pytest.mark.gpu
GUARD, FILL = 256, 0xA5


class Guarded:
    """An output with GUARD bytes on either side."""

    def __init__(self, shape, dtype):
        n = torch.empty(shape, dtype=dtype).numel() * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((n + 2 * GUARD,), FILL, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def untouched(self):
        return bool((self.raw[:GUARD] == FILL).all()) and bool((self.raw[-GUARD:] == FILL).all())


def outputs(M, K):
    codes = lambda m, k: (Guarded((m, k), torch.uint8), Guarded((k // 128, m), torch.float32))  # noqa: E731
    return {"z": (Guarded((M, K), torch.bfloat16),), "q": codes(M, K), "qT": codes(K, M), "qh": codes(M, K), "qy": codes(M, K)}


FIELDS = {"z": ("z",), "q": ("q", "s"), "qT": ("qT", "sT"), "qh": ("qh", "sh"), "qy": ("qy", "sy")}
SETS = [c for n in range(1, 6) for c in itertools.combinations(FIELDS, n) if set(c) & {"z", "q", "qT"}]


@pytest.mark.parametrize("K", [128, 640, 5120, 8192])
@pytest.mark.parametrize("post", [False, True])
def test_every_set_of_outputs(fp8lib, K, post):
    M = 128
    h, y, pre, post_g, _ = base.inputs(M, K, post, False)
    whole = fp8lib.residual_norm(h, y, pre, base.EPS, post_gamma=post_g, emit="bf16")
    want = {"z": (whole.z,), "q": fp8lib.quantize_1x128(whole.z)[:2], "qT": fp8lib.quantize_1x128(whole.z, dual=True)[2:],
            "qh": fp8lib.quantize_1x128(whole.h)[:2], "qy": fp8lib.quantize_1x128(y)[:2]}
    for chosen in SETS:
        out = outputs(M, K)
        fixed = {"h_out": Guarded((M, K), torch.bfloat16), "r_pre": Guarded((M,), torch.float32), "r_post": Guarded((M,), torch.float32)}
        a = _abi.ResidualNormArgs(h=h.data_ptr(), ldh=K, y=y.data_ptr(), ldy=K, pre_gamma=pre.data_ptr(), alpha=1.0, eps=base.EPS)
        if post:
            a.post_gamma = post_g.data_ptr()
        for f, g in fixed.items():
            if f != "r_post" or post:
                setattr(a, f, g.t.data_ptr())
        for name in chosen:
            for f, g in zip(FIELDS[name], out[name]):
                setattr(a, f, g.t.data_ptr())
        st = _abi.lib().fp8rl_residual_norm(ctypes.byref(a), M, K, torch.cuda.current_stream().cuda_stream)
        assert st == _abi.FP8RL_OK, chosen
        torch.cuda.synchronize()
        assert torch.equal(fixed["h_out"].t, whole.h) and torch.equal(fixed["r_pre"].t, whole.r_pre), chosen
        if post:
            assert torch.equal(fixed["r_post"].t, whole.r_post), chosen
        for g in fixed.values():
            assert g.untouched(), chosen
        for name, gs in out.items():
            for g, w in zip(gs, want[name]):
                assert g.untouched(), (chosen, name)
                if name in chosen:
                    assert torch.equal(g.t, w), (chosen, name)
                else:
                    assert bool((g.raw == FILL).all()), (chosen, name)
    assert fp8lib.check_status() == _abi.FP8RL_OK
