"""Plain 64-bit forms of windowed attention with sinks, and bounds of the kernels' rounding.

The bounds follow the roundings of the kernels, each at most half a step of
its type: probabilities in bf16 (2^-8) after a 2^x in fp16 (2^-11, and the
hardware's 2^x at 2^-9.9: together under 2^-9), the exponent in fp16 (2^-11 of
its magnitude, which lies within 8 of the distance to the row's maximum: the
reference may lag it by 8), scores in fp16 (2^-11 of each value rounded: the
two halves of a decode score and their sum), the output in bf16 (2^-8).  With
eps_j the relative error of probability j, an output o = sum_j p_j c_j is off
by at most sum_j p_j eps_j (|c_j| + |o|) + 2^-8 |o|; lse by sum_j p_j eps_j.
"""
import math

import numpy as np

SCALE = 1.0 / math.sqrt(192)
LN2 = math.log(2.0)


def seen_positions(p, window, sinks):
    """The positions a query at p sees, ascending."""
    return [j for j in range(p + 1) if j < sinks or j > p - window]


def _softmax(s):
    import torch
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(dim=-1, keepdim=True)
    return e / l, (m + torch.log(l)).squeeze(-1), (m - s) / LN2


def decode_row(q_abs, q_r, c, r):
    """One row's (o [H, 512], lse [H], bounds of both); c [n, 512], r [n, 64] the tokens it sees, 64 bits."""
    import torch
    half = [q_abs[:, 256 * i:256 * i + 256] @ c[:, 256 * i:256 * i + 256].T +
            q_r[:, 32 * i:32 * i + 32] @ r[:, 32 * i:32 * i + 32].T for i in range(2)]
    raw = half[0] + half[1]
    p, lse, dist = _softmax(raw * SCALE)
    eps = 2.0 ** -8 + 2.0 ** -9 + (dist + 8) * 2.0 ** -11 * LN2 + \
        (half[0].abs() + half[1].abs() + raw.abs()) * SCALE * 2.0 ** -11
    o = p @ c
    tol = (p * eps) @ c.abs() + o.abs() * (p * eps).sum(dim=-1, keepdim=True) + 2.0 ** -8 * o.abs()
    return o, lse, 1.05 * tol + 1e-6, 1.05 * (p * eps).sum(dim=-1) + 2.0 ** -22 * lse.abs() + 1e-6


def chunk(q_c, q_r, c, r, positions, key_positions, window, sinks, w_uk, w_uv):
    """A chunk's out [M, H, 128] and its bound; K_c and V_c are held in bf16 (2^-8 each)."""
    import torch
    M, H = q_c.shape[0], q_c.shape[1]
    out = torch.empty((M, H, 128), dtype=torch.float64, device=q_c.device)
    tol = torch.empty_like(out)
    hide = (key_positions[None] > positions[:, None]) | \
        ((key_positions[None] >= sinks) & (key_positions[None] <= positions[:, None] - window))
    for h in range(H):
        k, v = c @ w_uk[h].T, c @ w_uv[h]
        raw = q_c[:, h] @ k.T + q_r[:, h] @ r.T
        p, _, dist = _softmax((raw * SCALE).masked_fill(hide, -math.inf))
        eps = 2.0 ** -8 + 2.0 ** -9 + (dist.clamp(max=1e3) + 8) * 2.0 ** -11 * LN2 + raw.abs() * SCALE * 2.0 ** -11 + \
            (q_c[:, h].abs() @ k.abs().T) * SCALE * 2.0 ** -8
        o = p @ v
        out[:, h] = o
        tol[:, h] = (p * (eps + 2.0 ** -8)) @ v.abs() + o.abs() * (p * eps).sum(dim=-1, keepdim=True) + 2.0 ** -8 * o.abs()
    return out, 1.05 * tol + 1e-6


def bf16(rng, shape, std=1.0):
    from mla_latent_kv_02_gb300 import workloads as wl
    return wl.bf16_round(rng.standard_normal(shape, dtype=np.float32) * np.float32(std))
