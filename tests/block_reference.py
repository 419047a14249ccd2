"""Plain 64-bit definitions of the block operators (test infrastructure).

Written from the formulas: norms either side of a block with its gate and residual scale and
their gradients.  Where a result is a sum, the sum of its terms' magnitudes comes with it: the
bounds of the tests count roundings against that.
"""
from __future__ import annotations

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # 2^-8


def decode(saved):
    """Values in 64 bits of a saved tensor: bf16, or (codes u8 [M,K], scales f32 [K/128,M])."""
    if isinstance(saved, torch.Tensor):
        return saved.double()
    q, s = saved
    M, K = q.shape
    v = q.view(torch.float8_e4m3fn).double().view(M, K // 128, 128)
    return (v * s.double().t().unsqueeze(2)).reshape(M, K)


def rstd(x, eps):
    return (x.square().mean(1) + eps).rsqrt()


def residual_norm(h, y, pre, eps, post=None, gate=None, alpha=1.0):
    """(h', z, r_pre, r_post) without any rounding; 64-bit tensors."""
    n, rp = y, None
    if post is not None:
        rp = rstd(y, eps)
        n = y * rp[:, None] * post
    if gate is not None:
        n = n * gate
    h2 = h + alpha * n
    r = rstd(h2, eps)
    return h2, h2 * r[:, None] * pre, r, rp


def residual_norm_bwd(dz, dh, h, y, pre, r, post=None, rp=None, gate=None, alpha=1.0):
    """{name: (value, magnitude of its terms)}, from the definition's chain rule."""
    r = r[:, None]
    xh = h * r
    t = dz * pre
    dH = dh + r * (t - xh * (t * xh).mean(1, keepdim=True))
    mag = dh.abs() + r * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
    out = {"dh": (dH, mag), "dpre": ((dz * xh).sum(0), (dz * xh).abs().sum(0))}
    d, dm = alpha * dH, abs(alpha) * mag
    yh = y * rp[:, None] if post is not None else y
    if gate is not None:
        n = yh * post if post is not None else yh
        out["dgate"] = ((d * n).sum(0), (dm * n.abs()).sum(0))
        d, dm = d * gate, dm * gate.abs()
    if post is not None:
        out["dpost"] = ((d * yh).sum(0), (dm * yh.abs()).sum(0))
        u, um = d * post, dm * post.abs()
        rp = rp[:, None]
        d = rp * (u - yh * (u * yh).mean(1, keepdim=True))
        dm = rp * (um + yh.abs() * (um * yh.abs()).mean(1, keepdim=True))
    out["dy"] = (d, dm)
    return out


def decode_nvfp4(q, sf, g):
    """Values in 64 bits of NVFP4 rows: codes u8 [N,K/2], block scales in atoms of 128 rows x 4
    (row r of an atom at byte 16 (r % 32) + 4 (r / 32)), row scales [N]; N % 128 == 0."""
    N, K = q.shape[0], 2 * q.shape[1]
    c = torch.stack([q & 15, q >> 4], 2).view(N, K).long()
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=q.device)
    w = table[c & 7] * torch.where(c > 7, -1.0, 1.0).double()
    r, b = torch.arange(N, device=q.device)[:, None], torch.arange(K // 16, device=q.device)[None, :]
    at = 512 * ((r // 128) * (K // 64) + b // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4
    scale = sf.view(torch.float8_e4m3fn)[at].double()
    return w * scale.repeat_interleave(16, 1) * g.double()[:, None]
