"""The example's blocks as a whole: FP8 training with 8-bit checkpoints, rollout on 4-bit weights.

E4M3 with a scale per group has a relative error of about 2.6% (RMS of half a step of at most
2^-4); a product of two such operands 3.7%.  A gradient of the second block has gone through some
ten of them, of the first block twenty, adding in squares: 12% and 17%.  The test allows 25% of the
norm.  The rollout rounds to BF16 some six times a block, 2^-8 at most each: 2^-4 in all over two.
"""
import os
import sys

import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def stack64(x, first, blocks, alpha=1.0):
    """The same blocks in 64 bits; `blocks` hold 64-bit tensors."""
    h = x
    z = h * ref.rstd(h, 1e-5)[:, None] * first
    for b in blocks:
        g, u = (z @ b.w_gu.t()).chunk(2, dim=1)
        y = (torch.nn.functional.silu(g) * u) @ b.w_down.t()
        h, z, _, _ = ref.residual_norm(h, y, b.next_gamma, 1e-5, b.post_gamma, b.gate, alpha)
    return z


def setup(M, H, I, n):
    import mlp_block
    first, blocks = mlp_block.init(H, I, n, seed=3)
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((M, H), generator=gen, device="cuda").to(torch.bfloat16)
    dz = (1e-3 * torch.randn((M, H), generator=gen, device="cuda")).to(torch.bfloat16)
    return mlp_block, first, blocks, x, dz


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_training_gradients(fp8lib):
    mlp, first, blocks, x, dz = setup(384, 512, 768, 2)
    z, dx, grads, d_first = mlp.train_step(x, first, blocks, dz, alpha=0.5)
    assert fp8lib.check_status() == _abi.FP8RL_OK
    wide = [mlp.Block(*(t.double().requires_grad_() for t in b)) for b in blocks]
    x64, f64 = x.double().requires_grad_(), first.double().requires_grad_()
    z64 = stack64(x64, f64, wide, 0.5)
    (z64 * dz.double()).sum().backward()
    assert rel(z, z64.detach()) < 0.25
    assert rel(dx, x64.grad) < 0.25
    assert rel(d_first, f64.grad) < 0.25
    for g, b in zip(grads, wide):
        for name in mlp.Block._fields:
            assert rel(getattr(g, name), getattr(b, name).grad) < 0.25, name


@pytest.mark.parametrize("M", [1, 3, 16])
def test_rollout(fp8lib, M):
    mlp, first, blocks, x, _ = setup(16, 512, 768, 2)
    roll = mlp.Rollout(first, blocks)
    z = roll(x[:M])
    assert fp8lib.check_status() == _abi.FP8RL_OK
    exact = [mlp.Block(ref.decode_nvfp4(*gu), ref.decode_nvfp4(*dn), b.post_gamma.double(), b.gate.double(), b.next_gamma.double())
             for b, (gu, dn) in zip(blocks, roll.weights)]
    assert rel(z, stack64(x[:M].double(), first.double(), exact)) < 2.0 ** -4
