"""MLP blocks with a norm on either side, trained in FP8 with 8-bit checkpoints and rolled out
token by token on 4-bit weights.

A block adds to the residual stream h what its MLP makes of the normed stream z:

    y  = (silu(z Wg^T) * (z Wu^T)) Wd^T
    h' = h + alpha gate norm(y) post_gamma,     z' = norm(h') pre_gamma of the next block

Training keeps, per block and token, the codes of z in both layouts, the codes of the activation,
and three 8-bit checkpoints (gate_up output, h', y): no BF16 activation is saved.  Rollout runs
the same weights in NVFP4 with BF16 activations, up to 16 tokens at a time.

    python examples/mlp_block.py [tokens hidden intermediate blocks]
"""
from __future__ import annotations

import os
import sys
from typing import List, NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_x1_gb300.ops as fp8  # noqa: E402

EPS = 1e-5


class Block(NamedTuple):
    """BF16 master parameters: w_gu [2I,H], w_down [H,I], the others [H] (next_gamma belongs to
    the norm that follows the block)."""
    w_gu: torch.Tensor
    w_down: torch.Tensor
    post_gamma: torch.Tensor
    gate: torch.Tensor
    next_gamma: torch.Tensor


def init(H: int, I: int, blocks: int, seed: int = 0) -> tuple:
    """(first_gamma, [Block])"""
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    gain = lambda: (1 + 0.1 * rnd(H)).to(torch.bfloat16)  # noqa: E731
    made = [Block((rnd(2 * I, H) * H ** -0.5).to(torch.bfloat16), (rnd(H, I) * I ** -0.5).to(torch.bfloat16),
                  gain(), gain(), gain()) for _ in range(blocks)]
    return gain(), made


def train_step(x: torch.Tensor, first_gamma: torch.Tensor, blocks: List[Block], dz: torch.Tensor, alpha: float = 1.0):
    """Forward and backward of the stack: x bf16 [M,H] (M % 128 == 0), dz the gradient of the last
    norm's output.  Returns (z, dx, [gradients, a Block of them per block], d_first_gamma)."""
    q, s, qT, sT, rstd = fp8.rmsnorm_quant(x, first_gamma, EPS)
    saved, h = [], x
    for i, b in enumerate(blocks):
        q_gu, s_gu, q_guT = fp8.quantize_128x128(b.w_gu)
        q_dn, s_dn, q_dnT = fp8.quantize_128x128(b.w_down)
        gu = fp8.gemm_fwd(q, s, q_gu, s_gu)
        qa, sa, qaT, saT, q_ck, s_ck = fp8.silu_mul_quant_ckpt(gu)
        y = fp8.gemm_fwd(qa, sa, q_dn, s_dn)
        r = fp8.residual_norm(h, y, b.next_gamma, EPS, post_gamma=b.post_gamma, gate=b.gate, alpha=alpha,
                              emit="dual", checkpoint=True)
        saved.append((qT, sT, qaT, saT, q_ck, s_ck, r.h_ckpt, r.y_ckpt, r.r_pre, r.r_post, q_guT, s_gu, q_dnT, s_dn))
        h, q, s, qT, sT = r.h, r.q, r.s, r.qT, r.sT
    codes = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, 128)
    z = (codes * s.t().unsqueeze(2)).view(q.shape)

    grads, dh = [], None
    for b, kept in zip(reversed(blocks), reversed(saved)):
        qT, sT, qaT, saT, q_ck, s_ck, h_ck, y_ck, r_pre, r_post, q_guT, s_gu, q_dnT, s_dn = kept
        n = fp8.residual_norm_bwd(dz, dh, h_ck, y_ck, b.next_gamma, r_pre, post_gamma=b.post_gamma, r_post=r_post,
                                  gate=b.gate, alpha=alpha)
        qd, sd, qdT, sdT = fp8.quantize_1x128(n.dy, dual=True)
        d_act = fp8.gemm_dgrad(qd, sd, q_dnT, s_dn)
        dw_down = fp8.gemm_wgrad(qdT, sdT, qaT, saT)
        qd, sd, qdT, sdT = fp8.silu_mul_bwd_quant_ckpt(q_ck, s_ck, d_act)
        dz = fp8.gemm_dgrad(qd, sd, q_guT, s_gu)
        dw_gu = fp8.gemm_wgrad(qdT, sdT, qT, sT)
        dh = n.dh
        grads.append(Block(dw_gu, dw_down, n.dpost, n.dgate, n.dpre))
    dx, d_first = fp8.rmsnorm_bwd(x, first_gamma, rstd, dz)
    return z, (dx.float() + dh.float()).to(torch.bfloat16), grads[::-1], d_first


class Rollout:
    """The stack on NVFP4 weights for up to 16 tokens a call."""

    def __init__(self, first_gamma: torch.Tensor, blocks: List[Block], alpha: float = 1.0):
        self.first_gamma, self.blocks, self.alpha = first_gamma, blocks, alpha
        self.weights = [(fp8.quantize_nvfp4(b.w_gu), fp8.quantize_nvfp4(b.w_down)) for b in blocks]

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """x bf16 [M,H] -> the last norm's output bf16 [M,H]."""
        r = fp8.residual_norm(x, torch.zeros_like(x), self.first_gamma, EPS, emit="bf16")
        for b, (w_gu, w_down) in zip(self.blocks, self.weights):
            g, u = fp8.matvec_nvfp4(r.z, *w_gu).float().chunk(2, dim=1)
            a = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
            y = fp8.matvec_nvfp4(a, *w_down)
            r = fp8.residual_norm(r.h, y, b.next_gamma, EPS, post_gamma=b.post_gamma, gate=b.gate, alpha=self.alpha,
                                  emit="bf16")
        return r.z


def main(argv) -> None:
    M, H, I, n = (int(v) for v in argv) if argv else (1024, 1024, 2816, 2)
    first, blocks = init(H, I, n)
    x = torch.randn((M, H), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    dz = (1e-3 * torch.randn((M, H), generator=torch.Generator("cuda").manual_seed(2), device="cuda")).to(torch.bfloat16)
    z, dx, grads, _ = train_step(x, first, blocks, dz)
    roll = Rollout(first, blocks)
    one = torch.cat([roll(x[i:i + 1]) for i in range(4)])
    print(f"train: |z| {float(z.norm()):.1f}  |dx| {float(dx.float().norm()):.4f}  "
          f"|dW| {[round(float(g.w_gu.float().norm()), 4) for g in grads]}")
    far = float((one.float() - z[:4]).norm() / z[:4].norm())
    print(f"rollout of single tokens on 4-bit weights: {far:.3f} from the FP8 training forward")
    print("status", fp8.check_status())


if __name__ == "__main__":
    main(sys.argv[1:])
