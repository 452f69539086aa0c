"""The operators around an MLA layer's query and key preparation and its decoding, as cases to time and to compare.

  norm     RMS norms of the query heads and of the shared RoPE key, with the rotation in the same pass
  step     the same with its backward pass: the gradients of the queries, the key and both weights
  append   new latent rows and RoPE keys (normed and rotated on the way) into a paged cache that holds
           the latents in 4 bits, read back as the values that the cache stands for
  attend   attention of one or a few new tokens of each sequence over that cache, in the latent space

`own = False` computes them in their plain form (elementary torch operations in 32 bits); `own = True`
makes the framework's calls. The lengths, pages and row counts of a case come from the case alone, its
values from the seed.

The 4-bit format: a block of 16 latent values shares a scale, the smallest of the scale grid (3 fraction
bits, exponents -14 .. 13, below that steps of 2^-17) that brings the block's largest size to at most 6
scales; the codes are the multiples 0, 0.5, 1, 1.5, 2, 3, 4, 6 of the scale with a sign, to nearest, ties to
the even code. A code is 4 bits (the sign, then the index of the size), two in a byte, the even column's in
the low half; a scale is the upper 8 of an fp16's 15 bits below the sign. RoPE keys stay in the call's type.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 226  # 1.25 * 2^13: six of them are the largest value that the cache holds, 61440
EPS = 1e-6
THETA = 1e4

DSV3 = (512, 128, 64, 128)  # d_c, d_nope, d_rope, d_v
TINY = (64, 32, 16, 32)


# ---------------------------------------------------------------- cases
def _norm(name, op, dtype, B, S, n_h, d_nope, d_rope, **kw):
    c = dict(name=name, op=op, dtype=dtype, B=B, S=S, n_h=n_h, d_nope=d_nope, d_rope=d_rope, axes=1, interleaved=True,
             far=20000, key=True)
    c.update(kw)
    return c


def _cached(name, op, dtype, B, Sq, n_h, dims, page, shortest, longest, **kw):
    d_c, d_nope, d_rope, d_v = dims
    c = dict(name=name, op=op, dtype=dtype, B=B, Sq=Sq, n_h=n_h, d_c=d_c, d_nope=d_nope, d_rope=d_rope, d_v=d_v, page=page,
             shortest=shortest, longest=longest, empty=0, window=0, softcap=0.0, slopes=False, layout=1)
    c.update(kw)
    return c


def listed():
    return [
        # one new token's queries in each of 64 sequences, as a serving step norms them: latency
        _norm("norm_token_bf16", "norm", "bf16", 64, 1, 16, 128, 64, key=False),
        # the queries and keys of one rank of the 128-head sequence-parallel layer, three axes
        _norm("norm_shard_bf16", "norm", "bf16", 1, 2048, 128, 128, 64, axes=3, far=200000),
        # the same in training, with the gradients of the weights over all rows of all heads
        _norm("step_shard_bf16", "step", "bf16", 1, 2048, 128, 128, 64),
        # odd widths and lengths, halves layout, fp32
        _norm("step_odd_f32", "step", "f32", 2, 509, 3, 40, 24, interleaved=False, far=1000000),
        # one token appended to each of 64 sequences of a serving batch: latency
        _cached("append_token_bf16", "append", "bf16", 64, 1, 16, DSV3, 64, 0, 4096),
        # two prompts written at once, one shorter than the padded batch
        _cached("append_prompt_bf16", "append", "bf16", 2, 8192, 16, DSV3, 64, 0, 1000, layout=2),
        # the smallest: one token over a short history at the fp32 dimensions of the tests
        _cached("attend_tiny_f32", "attend", "f32", 3, 1, 4, TINY, 16, 1, 200),
        # a few tokens of one sequence of the mid-size layer: latency
        _cached("attend_few_bf16", "attend", "bf16", 1, 3, 16, DSV3, 64, 500, 700),
        # a serving batch at the mid-size layer's 16 heads, some sequences not begun: bound by the cache's bytes
        _cached("attend_batch_h16_bf16", "attend", "bf16", 64, 1, 16, DSV3, 64, 1000, 8192, empty=3),
        # the 128-head layer, long histories: bound by the products
        _cached("attend_batch_h128_bf16", "attend", "bf16", 24, 1, 128, DSV3, 64, 4000, 16384),
        # one long history alone: the work has to be split along it
        _cached("attend_long_h128_bf16", "attend", "bf16", 1, 1, 128, DSV3, 128, 100000, 131072),
        # drafted tokens checked together, capped scores, a window, odd pages
        _cached("attend_draft_cap_bf16", "attend", "bf16", 8, 5, 32, DSV3, 48, 200, 6000, window=4000, softcap=30.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "step", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "step"):
        c = _norm("", op, dtype, rng.choice([1, 1, 2, 3, 17]), 1, rng.choice([1, 2, 3, 7, 16, 40]),
                  rng.choice([0, 128, 128, rng.randrange(1, 130)]), rng.choice([2 * rng.randrange(1, 65), 64, 64]),
                  axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.5, far=_log_int(rng, 1, 2000000))
        c["S"] = _log_int(rng, 1, 2048 // c["B"])
        c["key"] = op == "step" or rng.random() < 0.7
    else:
        dims = DSV3 if dtype == "bf16" else (rng.randrange(1, 100), rng.randrange(1, 65), 2 * rng.randrange(1, 17), rng.randrange(1, 81))
        B = _log_int(rng, 1, 48)
        longest = _log_int(rng, 1, 1024 if dtype == "f32" else 8192)
        c = _cached("", op, dtype, B, 1, rng.choice([1, 2, 3, 5, 16, 24] if dtype == "bf16" else [1, 2, 3, 5]), dims,
                    rng.choice([1, 16, 64, 64, 128, rng.randrange(2, 200)]), rng.randrange(0, longest + 1), longest,
                    layout=rng.randrange(1, 1 << 20))
        if op == "append":
            c["Sq"] = rng.choice([1, 1, _log_int(rng, 1, 256)])
        else:
            c["Sq"] = rng.choice([1, 1, 1, 2, 4, rng.randrange(3, 14)])
            c["empty"] = rng.choice([0, 0, rng.randrange(0, B + 1)])
            c["window"] = rng.choice([0, 0, _log_int(rng, 1, longest)])
            c["softcap"] = rng.choice([0.0, 0.0, 5.0, 30.0])
            c["slopes"] = rng.random() < 0.25
    del c["name"]
    return c


# ---------------------------------------------------------------- layouts (from the case alone)
def _lengths(case):
    """Cached tokens of each sequence: for attend with the new ones, for append before them."""
    rng = random.Random(case["layout"])
    n = [rng.randint(case["shortest"], case["longest"]) for _ in range(case["B"])]
    for b in range(min(case["empty"], case["B"])):
        n[-1 - b] = 0
    return n


def _counts(case):
    """Rows of the padded batch that are appended to each sequence."""
    rng = random.Random(case["layout"] + 1)
    return [case["Sq"] if case["Sq"] == 1 else rng.randint(case["Sq"] // 2, case["Sq"]) for _ in range(case["B"])]


def _pages(case):
    """The table of pages [B, most pages of a sequence] (those past a sequence's end are -1), and the pages of the pool."""
    rng = random.Random(case["layout"] + 2)
    ends = [n + (case["Sq"] if case["op"] == "append" else 0) for n in _lengths(case)]
    need = [-(-n // case["page"]) for n in ends]
    total = sum(need) + 3
    ids = rng.sample(range(total), total)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (max(1, *need, 1) - n))
        at += n
    return table, total


def _sections(case):
    n, a = case["d_rope"] // 2, case["axes"]
    base = [n // a] * a
    base[-1] += n - sum(base)
    return base


def _bounds_np(case):
    """First visible key and one past the last of each query row."""
    n = np.asarray(_lengths(case))
    pos = n[:, None] - case["Sq"] + np.arange(case["Sq"])
    hi = np.maximum(pos + 1, 0)
    return (np.maximum(pos - case["window"] + 1, 0) if case["window"] else np.zeros_like(hi)), hi


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _dtype(case)
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dt)

    st = {"case": case}
    if case["op"] in ("norm", "step"):
        B, S, n_h, d = case["B"], case["S"], case["n_h"], case["d_nope"] + case["d_rope"]
        # rows of different size, as projections of tokens have; weights around 1
        st["q"] = normal(B, S, n_h, d) * torch.exp2(torch.randint(-3, 4, (B, S, n_h, 1), generator=g, device=dev)).to(dt)
        st["w_q"] = normal(d, std=0.2, mean=1.0)
        st["k_rope"] = normal(B, S, case["d_rope"], std=3.0) if case["key"] else None
        st["w_k"] = normal(case["d_rope"], std=0.2, mean=1.0) if case["key"] else None
        st["pos"] = torch.randint(0, case["far"], (case["axes"], B, S), generator=g, device=dev, dtype=torch.int32)
        st["sections"] = _sections(case)
        if case["op"] == "step":
            st["dq"], st["dk"] = normal(B, S, n_h, d), normal(B, S, case["d_rope"])
        return st
    B, Sq, d_c = case["B"], case["Sq"], case["d_c"]
    table, total = _pages(case)
    st["table"] = torch.tensor(table, dtype=torch.int32, device=dev)
    st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    # the pool as a running server has it: earlier tokens' latents everywhere
    rows = total * case["page"]
    codes, scales = _plain_encode(torch.randn(rows, d_c, generator=g, device=dev))
    st["codes"] = codes.view(total, case["page"], -1)
    st["scales"] = scales.view(total, case["page"], -1)
    st["keys"] = normal(total, case["page"], case["d_rope"])
    if case["op"] == "append":
        st["c_kv"] = normal(B, Sq, d_c)
        st["k_rope"] = normal(B, Sq, case["d_rope"], std=2.0)
        st["w_k"] = normal(case["d_rope"], std=0.2, mean=1.0)
        st["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
        return st
    n_h = case["n_h"]
    st["q"] = normal(B, Sq, n_h, case["d_nope"] + case["d_rope"], std=1.5)
    st["W_UK"] = normal(d_c, n_h * case["d_nope"], std=d_c ** -0.5)
    st["W_UV"] = normal(d_c, n_h * case["d_v"], std=d_c ** -0.5)
    st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / n_h) for h in range(n_h)], dtype=torch.float32,
                                device=dev) if case["slopes"] else None
    st["key_lo"] = torch.from_numpy(_bounds_np(case)[0].astype(np.int32)).to(dev) if case["window"] else None
    return st


# ---------------------------------------------------------------- plain forms
def _plain_encode(x):
    """(codes uint8 [rows, ceil(cols / 2)], scales uint8 [rows, ceil(cols / 16)]) of x [rows, cols]."""
    x = x.float()
    cols = x.shape[1]
    blocks = torch.nn.functional.pad(x, (0, -cols % BLOCK)).unflatten(1, (-1, BLOCK))
    grid = (torch.arange(TOP_SCALE + 1, device=x.device) << 7).to(torch.int16).view(torch.float16).float()
    top = blocks.abs().amax(-1)
    scale = torch.bucketize(top, 6.0 * grid, out_int32=True).clamp(max=TOP_SCALE)  # the first with top <= 6 grid
    a, s = blocks.abs(), grid[scale.long()][..., None]
    # halves between neighbouring sizes are exact multiples of the scale; a tie goes to the even code
    code = ((a > 0.25 * s).int() + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s) + (a >= 3.5 * s)
            + (a > 5.0 * s))
    code = torch.where(s > 0, code, 0) + 8 * (blocks < 0)
    code = code.flatten(1)[:, :cols]
    code = torch.nn.functional.pad(code, (0, cols % 2)).unflatten(1, (-1, 2))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), scale.to(torch.uint8)


def _plain_decode(codes, scales, cols):
    """The values [..., cols] of codes and scales, in 32 bits."""
    sizes = torch.tensor(SIZES + tuple(-v for v in SIZES), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :cols]
    s = (scales.int() << 7).to(torch.int16).view(torch.float16).float()
    return sizes[c.long()] * torch.repeat_interleave(s, BLOCK, -1)[..., :cols]


def _plain_rotation(pos, sections, d_rope, theta):
    """cos and sin [B, S, pairs] of the angles, taken in 64 bits."""
    n = d_rope // 2
    freq = theta ** (-torch.arange(n, dtype=torch.float64, device=pos.device) / n)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=pos.device),
                                   torch.tensor(sections, device=pos.device))
    ang = pos.double()[axis].permute(1, 2, 0) * freq
    return torch.cos(ang).float(), torch.sin(ang).float()


def _turn(x, cos, sin, interleaved):
    n = x.shape[-1] // 2
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :n], x[..., n:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_norm(x, w):
    """(x / rms(x), its product with w, 1 / rms(x)) in 32 bits."""
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, x * r * w.float(), r


def _plain_norm_rope(case, st):
    cos, sin = _plain_rotation(st["pos"], st["sections"], case["d_rope"], THETA)
    dn, dt = case["d_nope"], st["q"].dtype
    _, y, _ = _plain_norm(st["q"], st["w_q"])
    res = {"q": torch.cat([y[..., :dn], _turn(y[..., dn:], cos[:, :, None], sin[:, :, None], case["interleaved"])],
                          -1).to(dt)}
    if st["k_rope"] is not None:
        res["k_rope"] = _turn(_plain_norm(st["k_rope"], st["w_k"])[1], cos, sin, case["interleaved"]).to(dt)
    return res


def _plain_norm_back(x, w, dy):
    """The gradients of x and w from that of the normed rows, dy in 32 bits."""
    xh, _, r = _plain_norm(x, w)
    g = dy * w.float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dy * xh).flatten(0, -2).sum(0, dtype=torch.float64).to(w.dtype)


def _plain_norm_rope_back(case, st):
    cos, sin = _plain_rotation(st["pos"], st["sections"], case["d_rope"], THETA)
    dn, z = case["d_nope"], st["dq"].float()
    dy = torch.cat([z[..., :dn], _turn(z[..., dn:], cos[:, :, None], -sin[:, :, None], case["interleaved"])], -1)
    dq, dw_q = _plain_norm_back(st["q"], st["w_q"], dy)
    dk, dw_k = _plain_norm_back(st["k_rope"], st["w_k"], _turn(st["dk"].float(), cos, -sin, case["interleaved"]))
    return {"dq": dq, "dk_rope": dk, "dw_q": dw_q, "dw_k": dw_k}


def _slots(table, page, at):
    """Rows of the pool (flattened) that hold the positions `at` [B, n] of each sequence."""
    at = at.clamp(min=0, max=table.shape[1] * page - 1)
    return torch.gather(table.long(), 1, at // page).clamp(min=0) * page + at % page


def _plain_append(case, st):
    B, Sq, d_c = case["B"], case["Sq"], case["d_c"]
    i = torch.arange(Sq, device=st["table"].device)
    at = st["lengths"].long()[:, None] + i
    written = i < st["counts"][:, None]
    cos, sin = _plain_rotation(at[None], [case["d_rope"] // 2], case["d_rope"], THETA)
    keys = _turn(_plain_norm(st["k_rope"], st["w_k"])[1], cos, sin, True).to(_dtype(case))
    codes, scales = _plain_encode(st["c_kv"].reshape(B * Sq, d_c))
    slot = _slots(st["table"], case["page"], at)
    to = slot[written]
    st["codes"].flatten(0, 1)[to] = codes.view(B, Sq, -1)[written]
    st["scales"].flatten(0, 1)[to] = scales.view(B, Sq, -1)[written]
    st["keys"].flatten(0, 1)[to] = keys[written]
    c = _plain_decode(st["codes"].flatten(0, 1)[slot], st["scales"].flatten(0, 1)[slot], d_c)
    return {"c_kv": (c * written[..., None]).to(_dtype(case)), "k_rope": st["keys"].flatten(0, 1)[slot] * written[..., None]}


def _plain_attend(case, st):
    B, Sq, n_h, dn, dr, d_c = (case[k] for k in ("B", "Sq", "n_h", "d_nope", "d_rope", "d_c"))
    n = st["lengths"].long()
    j = torch.arange(st["table"].shape[1] * case["page"], device=n.device)[:max(_lengths(case) + [1])]
    slot = _slots(st["table"], case["page"], j.expand(B, -1))
    there = (j < n[:, None])[..., None]
    c = torch.where(there, _plain_decode(st["codes"].flatten(0, 1)[slot], st["scales"].flatten(0, 1)[slot], d_c), 0.0)
    keys = torch.where(there, st["keys"].flatten(0, 1)[slot].float(), 0.0)
    q = st["q"].float()
    q_lat = (q[..., :dn].reshape(B * Sq, n_h, dn).transpose(0, 1)
             @ st["W_UK"].float().view(d_c, n_h, dn).permute(1, 2, 0))  # [n_h, B Sq, d_c]
    q_lat = q_lat.transpose(0, 1).reshape(B, Sq * n_h, d_c)
    s = (q_lat @ c.transpose(1, 2) + q[..., dn:].reshape(B, Sq * n_h, dr) @ keys.transpose(1, 2)) * (dn + dr) ** -0.5
    s = s.view(B, Sq, n_h, -1)
    if case["softcap"]:
        s = torch.tanh(s / case["softcap"]) * case["softcap"]
    pos = n[:, None] - Sq + torch.arange(Sq, device=n.device)
    if st["slopes"] is not None:
        s = s - st["slopes"][:, None] * (pos[:, :, None, None] - j).abs()
    seen = j <= pos[..., None]
    if st["key_lo"] is not None:
        seen = seen & (j >= st["key_lo"][..., None])
    s = s.masked_fill(~seen[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    P = torch.exp(s - top)
    total = P.sum(-1, keepdim=True)
    ctx = P.view(B, Sq * n_h, -1) @ c / torch.where(total == 0, 1.0, total).view(B, Sq * n_h, 1)
    out = (ctx.view(B * Sq, n_h, d_c).transpose(0, 1)
           @ st["W_UV"].float().view(d_c, n_h, case["d_v"]).transpose(0, 1))  # [n_h, B Sq, d_v]
    return {"out": out.transpose(0, 1).reshape(B, Sq, n_h, case["d_v"]).to(_dtype(case))}


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "append":
        return _plain_append(case, state)
    if case["op"] == "attend":
        return _plain_attend(case, state)
    res = _plain_norm_rope(case, state)
    if case["op"] == "step":
        res.update(_plain_norm_rope_back(case, state))
    return res


def _own(case, st):
    from mla_attention_sequence_gb300 import laga
    if case["op"] in ("norm", "step"):
        kw = dict(eps=EPS, sections=st["sections"], theta=THETA, interleaved=case["interleaved"])
        q, k = laga.norm_rope(st["q"], st["k_rope"], st["pos"], st["w_q"], st["w_k"], **kw)
        res = {"q": q} if k is None else {"q": q, "k_rope": k}
        if case["op"] == "step":
            res.update(laga.norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k_rope"], st["pos"], st["w_q"], st["w_k"],
                                          **kw))
        return res
    cache = laga.Cache4(st["codes"], st["scales"], st["keys"], case["d_c"])
    if case["op"] == "append":
        laga.cache4_append(cache, st["c_kv"], st["k_rope"], st["table"], st["lengths"], counts=st["counts"],
                           k_weight=st["w_k"], eps=EPS, theta=THETA)
        c, k = laga.cache4_read(cache, st["table"], st["lengths"], case["Sq"], counts=st["counts"])
        return {"c_kv": c, "k_rope": k}
    out, _ = laga.cache4_fwd(st["q"], cache, st["W_UK"], st["W_UV"], st["table"], st["lengths"], key_lo=st["key_lo"],
                             softcap=case["softcap"], slopes=st["slopes"])
    return {"out": out}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "step"):
        rows, d = case["B"] * case["S"], case["d_nope"] + case["d_rope"]
        n = rows * (case["n_h"] * d + (case["d_rope"] if case["key"] else 0))
        if case["op"] == "norm":
            return {"bytes": 2 * n * e + 4 * case["axes"] * rows + e * d, "flops": 6 * n}
        # forward: rows in and out; backward: rows and their gradients in, gradients out
        return {"bytes": 5 * n * e + 8 * case["axes"] * rows + 2 * e * (d + case["d_rope"]), "flops": 20 * n}
    d_c, dr = case["d_c"], case["d_rope"]
    row = -(-d_c // 2) + -(-d_c // BLOCK) + dr * e  # a cached token
    if case["op"] == "append":
        n = sum(_counts(case))
        # rows in, cache rows out; the cache rows in again, values out for the whole padded batch
        return {"bytes": n * (e * (d_c + dr) + 2 * row) + case["B"] * case["Sq"] * e * (d_c + dr), "flops": 12 * n * (d_c + dr)}
    B, Sq, n_h, dn, dv = (case[k] for k in ("B", "Sq", "n_h", "d_nope", "d_v"))
    lo, hi = _bounds_np(case)
    pairs = int(np.maximum(hi - lo, 0).sum())
    tokens = int(sum(max(0, h.max() - l.min()) for l, h in zip(lo, hi)))
    weights = d_c * n_h * (dn + dv)
    # in the latent space, or with K and V rebuilt for the tokens that are seen: whichever is less
    latent = 2 * pairs * n_h * (2 * d_c + dr) + 2 * B * Sq * weights
    rebuilt = 2 * pairs * n_h * (dn + dr + dv) + 2 * tokens * weights
    return {"bytes": tokens * row + e * (weights + B * Sq * n_h * (dn + dr + dv)),
            "flops": min(latent, rebuilt)}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "step"):
        return _exact_norm(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_attend(case, st)


def _exact_turns(case, pos, sections):
    """e^(i angle) per row and pair, as numpy complex numbers."""
    n = case["d_rope"] // 2
    axis = np.concatenate([np.full(s, a) for a, s in enumerate(sections)])
    pos = pos.cpu().numpy().astype(np.float64)
    return torch.from_numpy(np.exp(1j * np.stack([pos[axis[i]] * THETA ** (-i / n) for i in range(n)], -1)))


def _exact_pairs(x, interleaved):
    n = x.shape[-1] // 2
    return torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :n], x[..., n:])


def _exact_flat(z, interleaved):
    return torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _exact_norm(case, st):
    turn = _exact_turns(case, st["pos"], st["sections"]).to(st["q"].device)
    dn, il = case["d_nope"], case["interleaved"]
    leaf = {k: st[k].double().requires_grad_(True) for k in ("q", "w_q", "k_rope", "w_k") if st[k] is not None}
    with torch.set_grad_enabled(case["op"] == "step"):
        y = leaf["q"] / torch.sqrt((leaf["q"] ** 2).sum(-1, keepdim=True) / leaf["q"].shape[-1] + EPS) * leaf["w_q"]
        res = {"q": torch.cat([y[..., :dn], _exact_flat(_exact_pairs(y[..., dn:], il) * turn[:, :, None], il)], -1)}
        if st["k_rope"] is not None:
            k = leaf["k_rope"]
            k = k / torch.sqrt((k ** 2).sum(-1, keepdim=True) / k.shape[-1] + EPS) * leaf["w_k"]
            res["k_rope"] = _exact_flat(_exact_pairs(k, il) * turn, il)
        if case["op"] == "step":
            ((res["q"] * st["dq"].double()).sum() + (res["k_rope"] * st["dk"].double()).sum()).backward()
    res = {k: v.detach() for k, v in res.items()}
    if case["op"] == "step":
        res.update(dq=leaf["q"].grad, dk_rope=leaf["k_rope"].grad, dw_q=leaf["w_q"].grad, dw_k=leaf["w_k"].grad)
    return res


def _exact_values(codes, scales, cols):
    """The cache's values in numpy, from the bits: sign, size, and an fp16 whose lowest 7 bits are 0."""
    codes, scales = codes.cpu().numpy().astype(np.int64), scales.cpu().numpy().astype(np.int64)
    c = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), np.int64)
    c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
    e, m = scales // 8, scales % 8
    s = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 15), m / 8 * 2.0 ** -14)
    v = np.asarray(SIZES)[c % 8] * np.where(c >= 8, -1.0, 1.0)
    return (v[..., :cols].reshape(-1, cols) * np.repeat(s.reshape(-1, s.shape[-1]), BLOCK, 1)[:, :cols]).reshape(
        *codes.shape[:-1], cols)


def _exact_append(case, st):
    at = st["lengths"].long()[:, None] + torch.arange(case["Sq"], device=st["lengths"].device)
    turn = _exact_turns(case, at[None], [case["d_rope"] // 2]).to(at.device)
    k = st["k_rope"].double()
    k = k / torch.sqrt((k ** 2).sum(-1, keepdim=True) / k.shape[-1] + EPS) * st["w_k"].double()
    k = _exact_flat(_exact_pairs(k, True) * turn, True)
    # the latents: nearest multiples of the block's scale, block by block
    x = st["c_kv"].double()
    c = torch.zeros_like(x)
    grid = torch.tensor([m * 2.0 ** -17 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 18) for e in range(1, 29) for m in range(8)],
                        dtype=torch.float64, device=x.device)[:TOP_SCALE + 1]
    sizes = torch.tensor(SIZES, dtype=torch.float64, device=x.device)
    for b in range(0, case["d_c"], BLOCK):
        v = x[..., b:b + BLOCK]
        s = grid[torch.searchsorted(grid, v.abs().amax(-1) / 6.0).clamp(max=TOP_SCALE)][..., None]
        r = v.abs() / torch.where(s > 0, s, 1.0)
        far = (r[..., None] - sizes).abs()
        near = far.amin(-1, keepdim=True)
        tied = far == near  # two at most, neighbours: the even one
        even = torch.arange(8, device=x.device) % 2 == 0
        pick = torch.where(tied.sum(-1, keepdim=True) > 1, tied & even, tied).double().argmax(-1)
        c[..., b:b + BLOCK] = sizes[pick] * s * torch.sign(v)
    written = (torch.arange(case["Sq"], device=x.device) < st["counts"][:, None])[..., None]
    return {"c_kv": c * written, "k_rope": k * written}


def _exact_attend(case, st):
    B, Sq, n_h, dn, dv, d_c = (case[k] for k in ("B", "Sq", "n_h", "d_nope", "d_v", "d_c"))
    lengths = _lengths(case)
    if n_h * Sq * sum(lengths) * (2 * d_c + case["d_rope"]) > 1e11:  # 64-bit products: some 1e12 a second
        return None
    lo, hi = _bounds_np(case)
    table, _ = _pages(case)
    dev = st["q"].device
    out = torch.zeros(B, Sq, n_h, dv, dtype=torch.float64, device=dev)
    W_UK, W_UV = st["W_UK"].double().view(d_c, n_h, dn), st["W_UV"].double().view(d_c, n_h, dv)
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        ids = torch.tensor(table[b][:-(-n // case["page"])], device=dev)
        c = torch.from_numpy(_exact_values(st["codes"][ids], st["scales"][ids], d_c)).to(dev).flatten(0, 1)[:n]
        k = st["keys"][ids].double().flatten(0, 1)[:n]
        q = st["q"][b].double()
        for i in range(Sq):
            a, z = int(lo[b, i]), int(hi[b, i])
            if a >= z:
                continue
            s = torch.einsum("chd,hd->hc", W_UK, q[i, :, :dn]) @ c[a:z].T + q[i, :, dn:] @ k[a:z].T
            s = s / math.sqrt(dn + case["d_rope"])
            if case["softcap"]:
                s = case["softcap"] * torch.tanh(s / case["softcap"])
            if st["slopes"] is not None:
                s = s - st["slopes"].double()[:, None] * (z - 1 - torch.arange(a, z, device=dev)).abs()
            out[b, i] = torch.einsum("hc,chd->hd", torch.softmax(s, -1) @ c[a:z], W_UV)
    return {"out": out}
