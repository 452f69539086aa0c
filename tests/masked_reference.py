"""The packed-document operators in 64 bits, written from their definitions (test infrastructure)."""
import math

import numpy as np
import torch


def bounds(doc_starts, n_rows, S, q_offset=0, prefix=None, window=0, q_split=0, q_offset2=0):
    """key_lo, key_hi row by row, in plain Python."""
    B, n_docs = len(doc_starts), len(doc_starts[0]) - 1
    lo, hi = np.zeros((B, n_rows), np.int64), np.zeros((B, n_rows), np.int64)
    for b in range(B):
        for i in range(n_rows):
            p = q_offset2 + i - q_split if q_split and i >= q_split else q_offset + i
            for k in range(n_docs):
                a, z = doc_starts[b][k], doc_starts[b][k + 1]
                if a <= p < z:
                    last = min(z, S)
                    lo[b, i] = max(a, p - window + 1) if window else a
                    hi[b, i] = min(max(p + 1, a + (prefix[b][k] if prefix else 0)), last)
    return lo, hi


def positions(Sq, q_offset, q_split=0, q_offset2=0):
    i = torch.arange(Sq)
    return torch.where(i >= q_split, q_offset2 + i - q_split, q_offset + i) if q_split else q_offset + i


def visible(Sq, S, key_lo=None, key_hi=None, causal=True, q_offset=0, q_split=0, q_offset2=0, B=1):
    j = torch.arange(S)
    pos = positions(Sq, q_offset, q_split, q_offset2)
    seen = torch.ones(B, Sq, S, dtype=torch.bool)
    if key_lo is not None:
        seen &= j >= key_lo.cpu().long()[..., None]
    if key_hi is not None:
        seen &= j < key_hi.cpu().long()[..., None]
    if causal:
        seen &= j <= pos[:, None]
    return seen


def attention(x, seen, softcap=0.0, slopes=None, scale=None, pos=None, dout=None, lse=None, out=None):
    """x: q, c_kv, k_rope, W_UK, W_UV (any type; masked places must be finite). seen [B, Sq, S].
    Returns out, lse and, with dout, the gradients and "mag": each gradient's size when no
    cancellation with D is counted (what rounding errors are relative to). lse / out: the saved
    ones, for a backward that starts from them."""
    x = {k: v.double() for k, v in x.items()}
    B, Sq, n_h, d_qk = x["q"].shape
    S, d_rope = x["k_rope"].shape[1:]
    dn, d_v = d_qk - d_rope, x["W_UV"].shape[1] // n_h
    scale = scale or d_qk ** -0.5
    dev = x["q"].device
    seen = seen.to(dev)[:, None]
    K = torch.einsum("bsc,chd->bhsd", x["c_kv"], x["W_UK"].view(-1, n_h, dn))
    K = torch.cat([K, x["k_rope"][:, None].expand(B, n_h, S, d_rope)], -1)
    V = torch.einsum("bsc,chd->bhsd", x["c_kv"], x["W_UV"].view(-1, n_h, d_v))
    q = x["q"].transpose(1, 2)
    s = q @ K.transpose(2, 3) * scale
    factor = torch.ones_like(s)
    if softcap:
        t = torch.tanh(s / softcap)
        s, factor = softcap * t, 1 - t * t
    if slopes is not None:
        dist = (pos.to(dev)[:, None] - torch.arange(S, device=dev)).abs()
        s = s - slopes.double().to(dev)[:, None, None] * dist
    s = s.masked_fill(~seen, -math.inf)
    if lse is None:
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        total = torch.exp(s - top).sum(-1, keepdim=True)
        L = torch.log(total) + top
    else:
        L = lse.double()[..., None]
    P = torch.exp(s - torch.where(L == -math.inf, 0.0, L))
    o = (P @ V).transpose(1, 2)
    res = {"out": o, "lse": L[..., 0]}
    if dout is None:
        return res
    do = dout.double().transpose(1, 2)
    D = (do * (o if out is None else out.double()).transpose(1, 2)).sum(-1, keepdim=True)
    dP = do @ V.transpose(2, 3)
    dV = P.transpose(2, 3) @ do
    W = x["W_UK"].view(-1, n_h, dn), x["W_UV"].view(-1, n_h, d_v)

    def back(dS):
        dK = dS.transpose(2, 3) @ q
        return {"dq": (dS @ K).transpose(1, 2), "dk_rope": dK[..., dn:].sum(1),
                "dc_kv": torch.einsum("bhsd,chd->bsc", dK[..., :dn], W[0]) + torch.einsum("bhsd,chd->bsc", dV, W[1]),
                "dW_UK": torch.einsum("bsc,bhsd->chd", x["c_kv"], dK[..., :dn]).flatten(1),
                "dW_UV": torch.einsum("bsc,bhsd->chd", x["c_kv"], dV).flatten(1)}

    res.update(back(P * (dP - D) * factor * scale))
    res["mag"] = {k: float(v.norm()) for k, v in back(P * dP * factor * scale).items()}
    return res


def close(got, ref, tol, names=None):
    """Each tensor's error, as a 2-norm relative to the reference's (or its uncancelled size)."""
    bad = []
    for k in names or [n for n in ref if n in got]:
        a, r = got[k].double(), ref[k].double().to(got[k].device)
        if k == "lse":
            empty = r == -math.inf
            assert torch.equal(a == -math.inf, empty), "lse of empty rows"
            a, r = a[~empty], r[~empty]
        size = max(float(r.norm()), ref.get("mag", {}).get(k, 0.0))
        err = float((a - r).norm())
        if not err <= tol * size:
            bad.append(f"{k}: {err:.3e} > {tol:.1e} * {size:.3e}")
    assert not bad, "; ".join(bad)


def e4m3_values():
    """The value of each e4m3 code."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        f = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-f if c & 128 else f)
    return np.array(v)


def pack8(x):
    """codes' values and scale bytes of a 2-D array, block by block, from the table of e4m3 values."""
    table = e4m3_values()
    pos = table[:127]  # 0 .. 448, ascending
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    vals, scales = np.zeros_like(x), np.zeros((rows, -(-cols // 32)), np.int64)
    for r in range(rows):
        for k in range(scales.shape[1]):
            blk = x[r, 32 * k:32 * k + 32]
            fin = np.abs(blk[np.isfinite(blk)])
            top = fin.max() if fin.size else 0.0
            e = 0
            if top > 0:
                e = -127
                while top / 2.0 ** e > 448:
                    e += 1
            scales[r, k] = e + 127
            for c, v in enumerate(blk):
                if not np.isfinite(v):
                    vals[r, 32 * k + c] = math.nan
                    continue
                a = abs(v) / 2.0 ** e
                i = int(np.searchsorted(pos, a))
                i = min(i, 126)
                if i > 0:
                    down, up = a - pos[i - 1], pos[i] - a
                    if down < up or (down == up and (i - 1) % 2 == 0):
                        i -= 1
                vals[r, 32 * k + c] = math.copysign(pos[i], v)
    return vals, scales
