"""The backward's ring of rows and its column sums over many rows of a block, and repeat calls of the
training sizes.

The shapes give a block (152 or more of them) 17 to 108 rows, so every slot of the rings of three and four
is filled again many times; bounds as for the short shapes, whose column sums count up to 130 rows."""
import pytest
import torch

import test_gpu_residual_norm as base
from block_scaled_fp8_x1_gb300 import _abi, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("saved", ["bf16", "fp8"])
@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,K", [(2500, 8192), (2501, 5248), (8192, 4096), (20000, 640)])
def test_many_rows_a_block(fp8lib, M, K, post, gated, saved):
    base.test_backward(fp8lib, M, K, post, gated, saved)
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.parametrize("saved", ["bf16", "fp8"])
def test_training_size(fp8lib, saved):
    base.test_backward(fp8lib, 16384, 5120, True, True, saved)


def same(calls):
    first = calls()
    for _ in range(3):
        for a, b in zip(first, calls()):
            assert a is None or torch.equal(a, b)


def test_training_sizes_repeat_bit_for_bit(fp8lib):
    M, K, I = 16384, 5120, 27648
    h, y, pre, post, gate = base.inputs(M, K, True, True)

    def norm():
        r = fp8lib.residual_norm(h, y, pre, 1e-5, post_gamma=post, gate=gate, alpha=0.5, emit="dual", checkpoint=True)
        return (*r[:8], *r.h_ckpt, *r.y_ckpt)

    same(norm)
    gu = synth.normal_bf16((M, 2 * I), 1.0, 3, "cuda")
    dh = synth.normal_bf16((M, I), 1e-3, 4, "cuda")
    same(lambda: fp8lib.silu_mul_quant_ckpt(gu))
    ck = fp8lib.silu_mul_quant_ckpt(gu, dual=False)[4:]
    same(lambda: fp8lib.silu_mul_bwd_quant_ckpt(*ck, dh))
    assert fp8lib.check_status() == _abi.FP8RL_OK
