"""The norms with rotation and the paged 4-bit cache in 64 bits, written from their definitions (test infrastructure)."""
import math

import numpy as np
import torch

import masked_reference as ref

SIZES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TOP = 226


def scale_values():
    """The value of each scale byte: an fp16 whose lowest 7 bits are 0 (248 and up: not finite)."""
    e, m = np.arange(256) // 8, np.arange(256) % 8
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 15.0), m / 8 * 2.0 ** -14)
    v[248:] = math.nan
    return v


def encode(x):
    """(codes, scales, values) of x [rows, cols], value by value."""
    grid = scale_values()[:TOP + 1]
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes, scales = np.zeros((rows, (cols + 1) // 2), np.uint8), np.zeros((rows, -(-cols // 16)), np.uint8)
    vals = np.zeros_like(x)
    for r in range(rows):
        for k in range(scales.shape[1]):
            blk = x[r, 16 * k:16 * k + 16]
            if not np.isfinite(blk).all():
                scales[r, k], vals[r, 16 * k:16 * k + 16] = 255, math.nan
                continue
            e = min(int(np.searchsorted(6 * grid, np.abs(blk).max())), TOP)
            scales[r, k] = e
            for i, v in enumerate(blk):
                far = np.abs(SIZES * grid[e] - min(abs(v), 6 * grid[e]))  # past the largest: as the largest
                best = [c for c in range(8) if far[c] == far.min()] if grid[e] else [0]
                c = best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0]
                col = 16 * k + i
                codes[r, col // 2] |= (c + (8 if v < 0 else 0)) << (4 * (col % 2))
                vals[r, col] = math.copysign(SIZES[c] * grid[e], v)
    return codes, scales, vals


def decode(codes, scales, cols):
    """The values [..., cols] that a cache's bytes stand for (torch, 64 bits)."""
    c = torch.stack([codes.cpu() & 15, codes.cpu() >> 4], -1).flatten(-2)[..., :cols].long()
    v = torch.from_numpy(SIZES)[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    return v * torch.from_numpy(scale_values())[scales.cpu().long()].repeat_interleave(16, -1)[..., :cols]


def turn(x, pos, sections, theta, interleaved):
    """x [..., tokens.., (heads,) d_rope] turned by pos [axes, tokens..]."""
    n = x.shape[-1] // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = torch.stack([pos[int(axis[i])].double() * theta ** (-i / n) for i in range(n)], -1)
    while ang.dim() < x.dim():
        ang = ang.unsqueeze(-2)
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    a, b = a * c - b * s, a * s + b * c
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def norm(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def norm_rope(q, k, pos, wq, wk, eps, sections, theta, interleaved):
    dn = q.shape[-1] - 2 * sum(sections)
    y = norm(q, wq, eps)
    y = torch.cat([y[..., :dn], turn(y[..., dn:], pos, sections, theta, interleaved)], -1)
    return y, None if k is None else turn(norm(k, wk, eps), pos, sections, theta, interleaved)


def attend(q, values, keys, W_UK, W_UV, table, lengths, page, key_lo=None, key_hi=None, softcap=0.0, slopes=None,
           causal=True, scale=None):
    """out, lse from the pool's values [pages, page, d_c] and keys, sequence by sequence."""
    B, Sq, n_h, _ = q.shape
    outs, lses = [], []
    for b in range(B):
        n = int(lengths[b])
        d_v = W_UV.shape[1] // n_h
        if n <= 0:
            outs.append(torch.zeros(Sq, n_h, d_v, dtype=torch.float64))
            lses.append(torch.full((n_h, Sq), -math.inf, dtype=torch.float64))
            continue
        ids = table[b, :-(-n // page)].long().cpu()
        c, k = values[ids].flatten(0, 1)[:n], keys.cpu().double()[ids].flatten(0, 1)[:n]
        pos = n - Sq + torch.arange(Sq)
        j = torch.arange(n)
        seen = torch.ones(1, Sq, n, dtype=torch.bool)
        if causal:
            seen &= j <= pos[:, None]
        if key_lo is not None:
            seen &= j >= key_lo[b].cpu().long()[:, None]
        if key_hi is not None:
            seen &= j < key_hi[b].cpu().long()[:, None]
        x = dict(q=q[b:b + 1].cpu(), c_kv=c[None], k_rope=k[None], W_UK=W_UK.cpu(), W_UV=W_UV.cpu())
        r = ref.attention(x, seen, softcap, None if slopes is None else slopes.cpu(), scale, pos)
        outs.append(r["out"][0])
        lses.append(r["lse"][0])
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
