"""An expert layer with its norm and residual, trained in FP8 and rolled out a few tokens at a time
on the same FP8 weights.

    z   = norm(h) gamma
    k experts of a token by its router's scores, weights renormalised
    h'  = h + sum_j weight_j (silu(z Wg_e^T) * (z Wu_e^T)) Wd_e^T       over the token's experts e

Training sorts the (token, expert) pairs with every expert's rows at a multiple of 128 and keeps, per
pair, the 8-bit operands of the weight gradients; rollout sorts them without padding.

    python examples/expert_block.py [tokens hidden intermediate experts k]
"""
from __future__ import annotations

import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_x1_gb300.ops as fp8  # noqa: E402

EPS = 1e-5


class Experts(NamedTuple):
    """BF16 master parameters: router [E,H], w_gu [E 2I,H] and w_down [E H,I] (the experts' matrices
    one below the other), gamma [H]."""
    gamma: torch.Tensor
    router: torch.Tensor
    w_gu: torch.Tensor
    w_down: torch.Tensor


def init(H: int, I: int, E: int, seed: int = 0) -> Experts:
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return Experts((1 + 0.1 * rnd(H)).to(torch.bfloat16), (rnd(E, H) * H ** -0.5).to(torch.bfloat16),
                   (rnd(E * 2 * I, H) * H ** -0.5).to(torch.bfloat16), (rnd(E * H, I) * I ** -0.5).to(torch.bfloat16))


def _norm(h: torch.Tensor, gamma: torch.Tensor):
    r = fp8.residual_norm(h, torch.zeros_like(h), gamma, EPS, emit="bf16")
    return r.z, r.r_pre


def train_step(h: torch.Tensor, p: Experts, k: int, dout: torch.Tensor):
    """Forward and backward: h bf16 [M,H], dout the gradient of h'.  Returns (h', dh, gradients, the
    experts chosen)."""
    E = p.router.shape[0]
    z, rstd = _norm(h, p.gamma)
    logits = z.float() @ p.router.float().t()
    route = fp8.route_topk(logits, k)
    rows = fp8.expert_rows(route.index, E)
    q_gu, s_gu, q_guT = fp8.quantize_128x128(p.w_gu)
    q_dn, s_dn, q_dnT = fp8.quantize_128x128(p.w_down)

    qx, sx, qxT, sxT = fp8.expert_gather_quant(z, rows, dual=True)
    gu = fp8.gemm_experts_fwd(qx, sx, q_gu, s_gu, rows)
    qa, sa, qaT, saT = fp8.silu_mul_quant(gu)
    y = fp8.gemm_experts_fwd(qa, sa, q_dn, s_dn, rows)
    out = fp8.expert_combine(y, rows, route.weight, residual=h)

    qd, sd, qdT, sdT, dweight = fp8.expert_combine_bwd(dout, y, rows, route.weight)
    d_act = fp8.gemm_experts_dgrad(qd, sd, q_dnT, s_dn, rows)
    dw_down = fp8.gemm_experts_wgrad(qdT, sdT, qaT, saT, rows)
    qd, sd, qdT, sdT = fp8.silu_mul_bwd_quant(gu, d_act)
    dxp = fp8.gemm_experts_dgrad(qd, sd, q_guT, s_gu, rows)
    dw_gu = fp8.gemm_experts_wgrad(qdT, sdT, qxT, sxT, rows)
    dlogits = fp8.route_topk_bwd(dweight, logits, route.index)
    dz = fp8.expert_combine(dxp, rows, residual=(dlogits @ p.router.float()).to(torch.bfloat16))
    dh, dgamma = fp8.rmsnorm_bwd(h, p.gamma, rstd, dz)
    grads = Experts(dgamma, dlogits.t() @ z.float(), dw_gu.view_as(p.w_gu), dw_down.view_as(p.w_down))
    return out, (dh.float() + dout.float()).to(torch.bfloat16), grads, route.index


class Rollout:
    """The layer on the FP8 weights of training, for a few tokens a call."""

    def __init__(self, p: Experts, k: int):
        self.p, self.k = p, k
        self.router = p.router.float().t().contiguous()
        self.gu, self.down = fp8.quantize_128x128(p.w_gu, transpose=False), fp8.quantize_128x128(p.w_down, transpose=False)

    def __call__(self, h: torch.Tensor) -> torch.Tensor:
        z, _ = _norm(h, self.p.gamma)
        route = fp8.route_topk(z.float() @ self.router, self.k)
        rows = fp8.expert_rows(route.index, self.p.router.shape[0], align=1)
        q, s, _, _ = fp8.expert_gather_quant(z, rows)
        gu = fp8.gemm_experts_fwd(q, s, *self.gu[:2], rows)
        q, s, _, _ = fp8.silu_mul_quant(gu, dual=False)
        y = fp8.gemm_experts_fwd(q, s, *self.down[:2], rows)
        return fp8.expert_combine(y, rows, route.weight, residual=h)


def main(argv) -> None:
    M, H, I, E, k = (int(v) for v in argv) if argv else (1000, 1024, 640, 32, 4)
    p = init(H, I, E)
    h = torch.randn((M, H), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    dout = (1e-3 * torch.randn((M, H), generator=torch.Generator("cuda").manual_seed(2), device="cuda")).to(torch.bfloat16)
    out, dh, grads, index = train_step(h, p, k, dout)
    roll = Rollout(p, k)
    few = torch.cat([roll(h[:1]), roll(h[1:8])])
    print(f"train: |h'| {float(out.float().norm()):.1f}  |dh| {float(dh.float().norm()):.4f}  "
          f"|dW| {float(grads.w_gu.float().norm()):.4f}  tokens an expert {int(index.numel() / E)}")
    far = float((few.float() - out[:8].float()).norm() / (out[:8].float() - h[:8].float()).norm())
    print(f"rollout of 1 and 7 tokens: {far:.4f} from the training forward")
    print("status", fp8.check_status())


if __name__ == "__main__":
    main(sys.argv[1:])
