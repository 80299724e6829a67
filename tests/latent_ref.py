"""Plain 64-bit forms of the latent attention operators (torch, float64), for the tests. They
share no code with the library; each follows the definition in the public header."""
from __future__ import annotations

import math

import torch


def rotate(x, positions, inv_freq, magnitude, interleaved):
    """x [T, ..., P] in float64, its first 2 len(inv_freq) elements turned; also the size
    |x0| + |x1| behind each element."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = magnitude * angle.cos(), magnitude * angle.sin()
    while cos.dim() < x.dim():
        cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        i0 = torch.arange(half, device=x.device) * 2
        i1 = i0 + 1
    else:
        i0 = torch.arange(half, device=x.device)
        i1 = i0 + half
    y, size = x.clone(), x.abs()
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * cos - b * sin, b * cos + a * sin
    size[..., i0] = size[..., i1] = abs(magnitude) * (a.abs() + b.abs())
    return y, size


def normed(c, weight, eps):
    c = c.double()
    return c / (c.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def attend(q, keys, values, pos, scale, window=0, exists=None):
    """q [n, H, D], keys [H or 1, L, D], values [H or 1, L, V] in float64 (finite), row i at pos[i].
    Returns out [n, H, V], lse [n, H], and the sums sum_j w_j |v_j| and
    max_j |scale| sum_d |q_d k_d| that bound the error."""
    n, H, _ = q.shape
    L = keys.shape[1]
    j = torch.arange(L, device=q.device)
    seen = j[None, :] <= pos[:, None]
    if window:
        seen &= j[None, :] > pos[:, None] - window
    if exists is not None:
        seen &= exists[None, :]
    qh = q.permute(1, 0, 2)                                          # [H, n, D]
    z = scale * (qh @ keys.transpose(1, 2)).expand(H, n, L)
    z = z.masked_fill(~seen, -math.inf)
    reach = abs(scale) * (qh.abs() @ keys.abs().transpose(1, 2)).expand(H, n, L)
    reach = reach.masked_fill(~seen, 0).amax(-1) if L else torch.zeros(H, n).to(z)
    lse = torch.logsumexp(z, -1) if L else torch.full((H, n), -math.inf).to(z)
    w = (z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]).exp()
    out, size = w @ values, w @ values.abs()
    return out.permute(1, 0, 2), lse.T, size.permute(1, 0, 2), reach.T
