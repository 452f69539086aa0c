"""The training operators around packed documents, as cases to time and to compare.

Three groups of operators of an MLA training step:

  attention   masked attention over the rebuilt K/V (documents, prefixes, windows, capped
              scores, a bias by distance): the forward alone, the whole step with its
              gradients, and the backward that starts from an 8-bit checkpoint
  rope        rotary positions with several axes (time, height, width) on the queries and
              the shared key, forward and back
  pack        activation checkpoints in 8 bits: saving one, restoring one

`own = False` computes them in their plain form (elementary torch operations in 32 bits);
`own = True` makes the framework's calls. The document layout of a case comes from the case
alone, its values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

F8_MAX = 448.0  # largest e4m3 value
BLOCK = 32      # values that share one scale


# ---------------------------------------------------------------- cases
def _attn(name, op, dtype, B, Sq, S, n_h, dims, q_offset, docs, **kw):
    d_c, d_nope, d_rope, d_v = dims
    c = dict(name=name, op=op, dtype=dtype, B=B, Sq=Sq, S=S, n_h=n_h, d_c=d_c, d_nope=d_nope, d_rope=d_rope, d_v=d_v,
             q_offset=q_offset, docs=docs, pad=0, prefix=0.0, window=0, softcap=0.0, slopes=False, layout=1)
    c.update(kw)
    return c


DSV3 = (512, 128, 64, 128)
TINY = (64, 32, 16, 32)


def listed():
    return [
        # the smallest training step of the configurations, documents and capped scores, fp32
        _attn("step_tiny_f32", "step", "f32", 1, 256, 256, 4, TINY, 0, 3, softcap=30.0),
        # widths and lengths that fill no tile, prefix documents, a bias by distance, padded rows, fp32
        _attn("step_odd_f32", "step", "f32", 2, 509, 509, 3, (72, 40, 24, 56), 0, 4, pad=37, prefix=0.3, slopes=True),
        # a handful of query rows with a window, as a short last chunk of a sequence: latency
        _attn("fwd_few_rows_bf16", "fwd", "bf16", 1, 7, 519, 5, DSV3, 512, 1, window=200),
        # an evaluation pass over prefix documents with capped scores, forward only
        _attn("fwd_prefix_cap_bf16", "fwd", "bf16", 1, 4001, 4001, 16, DSV3, 0, 3, prefix=0.4, softcap=30.0),
        # the mid-size training configuration with packed documents and a bias by distance
        _attn("step_mid_bf16", "step", "bf16", 2, 4096, 4096, 16, DSV3, 0, 5, slopes=True),
        # the last rank of the 128-head sequence-parallel layer, one long document behind short ones
        _attn("step_shard_bf16", "step", "bf16", 1, 2048, 16384, 128, DSV3, 14336, 4, layout=4),
        # a backward that starts from the 8-bit checkpoint of q and out, odd length, padded rows
        _attn("packed_bwd_bf16", "packed_bwd", "bf16", 1, 2999, 2999, 32, DSV3, 0, 6, pad=55, softcap=50.0),
        # the same at the smallest training configuration, fp32
        _attn("packed_bwd_tiny_f32", "packed_bwd", "f32", 1, 256, 256, 4, TINY, 0, 2, slopes=True),
        # the rotation of one rank's queries and keys: 128 heads, three axes
        dict(name="rope_shard_bf16", op="rope", dtype="bf16", B=1, S=2048, n_h=128, d_nope=128, d_rope=64, axes=3,
             interleaved=True, inverse=False, theta=1e4, far=200000, layout=1),
        # the rotation's gradient at small odd sizes, one axis, far positions, halves layout
        dict(name="rope_back_f32", op="rope", dtype="f32", B=2, S=77, n_h=3, d_nope=32, d_rope=16, axes=1,
             interleaved=False, inverse=True, theta=5e5, far=1000000, layout=1),
        # one rank's queries saved in 8 bits
        dict(name="save_q_shard_bf16", op="save", dtype="bf16", rows=262144, cols=192, layout=1),
        # rows that end inside a block of 32, fp32, saved and restored
        dict(name="restore_odd_f32", op="restore", dtype="f32", rows=4093, cols=77, layout=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "step", "fwd", "fwd", "packed_bwd", "rope", "save", "restore"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    layout = rng.randrange(1, 1 << 20)
    if op in ("save", "restore"):
        cols = rng.choice([_log_int(rng, 1, 513), 64, 128, 192, 512])
        return dict(op=op, dtype=dtype, rows=min(_log_int(rng, 1, 262144), 50_000_000 // cols), cols=cols, layout=layout)
    if op == "rope":
        d_rope = rng.choice([2 * rng.randrange(1, 65), 64, 64])
        return dict(op=op, dtype=dtype, B=rng.choice([1, 1, 2, 3]), S=_log_int(rng, 1, 2048),
                    n_h=rng.choice([1, 2, 3, 7, 16, 40]), d_nope=rng.choice([0, 128, 128, rng.randrange(1, 130)]),
                    d_rope=d_rope, axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 1e6]), far=_log_int(rng, 1, 2000000),
                    layout=layout)
    if dtype == "f32":
        S = _log_int(rng, 16, 1024)
        n_h = rng.randrange(1, 7)
        dims = (rng.randrange(1, 100), rng.randrange(1, 65), rng.randrange(1, 33), rng.randrange(1, 81))
        B = rng.choice([1, 1, 2])
    else:
        S = _log_int(rng, 16, 8192)
        n_h = rng.choice([1, 2, 3, 5, 8, 16, 24])
        dims = DSV3
        B = rng.choice([1, 1, 2]) if S < 4096 else 1
    Sq = S if rng.random() < 0.5 else _log_int(rng, 1, S)
    c = _attn("", op, dtype, B, Sq, S, n_h, dims, S - Sq, rng.randrange(1, 9), layout=layout)
    c["pad"] = rng.choice([0, 0, rng.randrange(0, S - 15)])
    kind = rng.choice(["docs", "prefix", "window"])
    c["prefix"] = rng.choice([0.2, 0.5, 1.0]) if kind == "prefix" else 0.0
    c["window"] = _log_int(rng, 8, S) if kind == "window" else 0
    c["softcap"] = rng.choice([0.0, 0.0, 5.0, 30.0])
    c["slopes"] = rng.random() < 0.4
    del c["name"]
    return c


# ---------------------------------------------------------------- layouts (from the case alone)
def _documents(case):
    """(doc_starts [B][docs + 1], prefix lengths [B][docs]) of the packed sequences: documents of at
    least 9 tokens, then empty ones where fewer than `docs` fit, then the padding."""
    rng = random.Random(case["layout"])
    starts, prefixes = [], []
    for _ in range(case["B"]):
        end = case["S"] - case["pad"]
        cuts = sorted(rng.sample(range(1, max(1, end // 16)), min(case["docs"] - 1, max(0, end // 16 - 1))))
        s = [0] + [16 * c + rng.randrange(8) for c in cuts]
        s += [end] * (case["docs"] + 1 - len(s))
        starts.append(s)
        prefixes.append([int(case["prefix"] * (b - a)) for a, b in zip(s, s[1:])])
    return starts, prefixes


def _bounds_np(case):
    """First visible key and one past the last, per query row, in numpy."""
    starts, prefixes = _documents(case)
    pos = case["q_offset"] + np.arange(case["Sq"])
    lo, hi = np.zeros((case["B"], case["Sq"]), np.int64), np.zeros((case["B"], case["Sq"]), np.int64)
    for b in range(case["B"]):
        s = np.asarray(starts[b])
        d = np.searchsorted(s, pos, side="right") - 1
        inside = d < case["docs"]
        d = np.minimum(d, case["docs"] - 1)
        first, last, pre = s[d], s[d + 1], np.asarray(prefixes[b])[d]
        lo[b] = np.maximum(first, pos - case["window"] + 1) if case["window"] else first
        hi[b] = np.minimum(np.maximum(pos + 1, first + pre), last)
        lo[b][~inside] = 0
        hi[b][~inside] = 0
    return lo, hi


def _sections(case):
    """How many rotated pairs each axis has."""
    n, a = case["d_rope"] // 2, case["axes"]
    base = [n // a] * a
    base[-1] += n - sum(base)
    return base


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _dtype(case)
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    st = {"case": case}
    if case["op"] in ("save", "restore"):
        # activations: rows of very different size, as tokens have
        size = torch.exp2(torch.randint(-6, 4, (case["rows"], 1), generator=g, device=dev).float())
        st["x"] = (torch.randn(case["rows"], case["cols"], generator=g, device=dev) * size).to(dt)
    elif case["op"] == "rope":
        B, S = case["B"], case["S"]
        st["q"] = normal(B, S, case["n_h"], case["d_nope"] + case["d_rope"])
        st["k_rope"] = normal(B, S, case["d_rope"])
        st["pos"] = torch.randint(0, case["far"], (case["axes"], B, S), generator=g, device=dev, dtype=torch.int32)
        st["sections"] = _sections(case)
    else:
        B, Sq, S, n_h = case["B"], case["Sq"], case["S"], case["n_h"]
        w_std = case["d_c"] ** -0.5
        st["q"] = normal(B, Sq, n_h, case["d_nope"] + case["d_rope"])
        st["c_kv"] = normal(B, S, case["d_c"])
        st["k_rope"] = normal(B, S, case["d_rope"])
        st["W_UK"] = normal(case["d_c"], n_h * case["d_nope"], std=w_std)
        st["W_UV"] = normal(case["d_c"], n_h * case["d_v"], std=w_std)
        st["dout"] = normal(B, Sq, n_h, case["d_v"])
        starts, prefixes = _documents(case)
        st["doc_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        st["prefix"] = torch.tensor(prefixes, dtype=torch.int32, device=dev) if case["prefix"] else None
        # slopes in a geometric row, 2^(-8 (h + 1) / n_h)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / n_h) for h in range(n_h)], dtype=torch.float32,
                                    device=dev) if case["slopes"] else None
        if case["op"] == "packed_bwd":
            # the forward that ran earlier has left its statistics, and q and out as checkpoints
            out, st["lse"] = _plain_forward(case, st)
            st["q8"], st["q8_scales"] = _plain_save(st.pop("q"))
            st["out8"], st["out8_scales"] = _plain_save(out)
    return st


# ---------------------------------------------------------------- plain forms
def _plain_bounds(case, doc_starts, prefix):
    """key_lo, key_hi [B, Sq]: the keys of the row's own document that it sees."""
    pos = case["q_offset"] + torch.arange(case["Sq"], device=doc_starts.device)
    d = (pos[None, :, None] >= doc_starts[:, None, :].long()).sum(-1) - 1
    inside = d < case["docs"]
    d = d.clamp(max=case["docs"] - 1)
    first, last = torch.gather(doc_starts.long(), 1, d), torch.gather(doc_starts.long(), 1, d + 1)
    lo = torch.maximum(first, pos - case["window"] + 1) if case["window"] else first
    hi = pos[None] + 1
    if prefix is not None:
        hi = torch.maximum(hi, first + torch.gather(prefix.long(), 1, d))
    hi = torch.minimum(hi, last)
    return torch.where(inside, lo, 0), torch.where(inside, hi, 0)


def _plain_scores(case, st, q):
    """K and V [B, h, S, .], the masked scores s [B, h, Sq, S] and their tanh (or None)."""
    B, Sq, S, n_h, dn = case["B"], case["Sq"], case["S"], case["n_h"], case["d_nope"]
    c = st["c_kv"].float()
    K = (c @ st["W_UK"].float()).view(B, S, n_h, dn).transpose(1, 2)
    V = (c @ st["W_UV"].float()).view(B, S, n_h, case["d_v"]).transpose(1, 2)
    K = torch.cat([K, st["k_rope"].float()[:, None].expand(B, n_h, S, case["d_rope"])], -1)
    s = (q @ K.transpose(2, 3)).mul_((dn + case["d_rope"]) ** -0.5)
    th = None
    if case["softcap"]:
        th = s.div_(case["softcap"]).tanh_()
        s = th * case["softcap"]
    pos = case["q_offset"] + torch.arange(Sq, device=q.device)
    key = torch.arange(S, device=q.device)
    if st["slopes"] is not None:
        s.sub_(st["slopes"][:, None, None] * (pos[:, None] - key).abs().float())
    lo, hi = _plain_bounds(case, st["doc_starts"], st["prefix"])
    seen = (key >= lo[..., None]) & (key < hi[..., None])
    s.masked_fill_(~seen[:, None], -math.inf)
    return K, V, s, th


def _plain_softmax(s):
    """P over s's memory, and lse [B, h, Sq, 1] (-inf, and a row of zeros, where nothing is seen)."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    P = s.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    P.div_(torch.where(total == 0, 1.0, total))
    return P, total.log() + top


def _plain_forward(case, st):
    _, V, s, _ = _plain_scores(case, st, st["q"].float().transpose(1, 2))
    P, lse = _plain_softmax(s)
    return (P @ V).transpose(1, 2).contiguous().to(_dtype(case)), lse[..., 0]


def _plain_backward(case, st, q, out, K, V, P, th):
    """The gradients of <dout, out> through P, the scores and the rebuild."""
    dt, dn, B, S, n_h = _dtype(case), case["d_nope"], case["B"], case["S"], case["n_h"]
    dout = st["dout"].float().transpose(1, 2)
    D = (dout * out).sum(-1, keepdim=True)
    dV = P.transpose(2, 3) @ dout
    dS = (dout @ V.transpose(2, 3)).sub_(D).mul_(P).mul_((dn + case["d_rope"]) ** -0.5)
    if th is not None:
        dS.mul_(th.square_().neg_().add_(1.0))
    dq = (dS @ K).transpose(1, 2).contiguous()
    dK = dS.transpose(2, 3) @ q
    dk_rope = dK[..., dn:].sum(1)
    dK = dK[..., :dn].transpose(1, 2).reshape(B * S, n_h * dn)
    dV = dV.transpose(1, 2).reshape(B * S, n_h * case["d_v"])
    c = st["c_kv"].float().view(B * S, -1)
    dc = dK @ st["W_UK"].float().t() + dV @ st["W_UV"].float().t()
    return dict(dq=dq.to(dt), dk_rope=dk_rope.to(dt), dc_kv=dc.view(B, S, -1).to(dt), dW_UK=(c.t() @ dK).to(dt),
                dW_UV=(c.t() @ dV).to(dt))


def _plain_attention(case, st):
    if case["op"] == "fwd":
        return {"out": _plain_forward(case, st)[0]}
    if case["op"] == "step":
        q = st["q"].float().transpose(1, 2)
        K, V, s, th = _plain_scores(case, st, q)
        P, _ = _plain_softmax(s)
        out = P @ V
        return {"out": out.transpose(1, 2).contiguous().to(_dtype(case)),
                **_plain_backward(case, st, q, out, K, V, P, th)}
    # the backward from the checkpoints: P = exp(s - lse) with the saved lse at the restored q
    q = _plain_restore(st["q8"], st["q8_scales"]).transpose(1, 2)
    out = _plain_restore(st["out8"], st["out8_scales"]).transpose(1, 2)
    K, V, s, th = _plain_scores(case, st, q)
    lse = st["lse"][..., None]
    P = s.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    return _plain_backward(case, st, q, out, K, V, P, th)


def _plain_rope(case, st):
    """Pair i turns by pos[axis(i)] * theta^(-2 i / d_rope); angles in 64 bits."""
    n = case["d_rope"] // 2
    dev = st["q"].device
    freq = case["theta"] ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=dev), torch.tensor(st["sections"], device=dev))
    ang = st["pos"].double()[axis].permute(1, 2, 0) * freq  # [B, S, n]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if case["inverse"]:
        sin = -sin

    def turn(x, cos, sin):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        a, b = x[..., :n], x[..., n:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    q, dn = st["q"], case["d_nope"]
    rot = turn(q[..., dn:], cos[:, :, None], sin[:, :, None]).to(q.dtype)
    return {"q": torch.cat([q[..., :dn], rot], -1), "k_rope": turn(st["k_rope"], cos, sin).to(q.dtype)}


def _plain_save(x):
    """(codes float8_e4m3fn [.., cols], biased scale exponents uint8 [.., blocks]): a block of 32
    shares the smallest power of two that brings its largest finite size to at most 448."""
    x = x.float()
    pad = -x.shape[-1] % BLOCK
    blocks = torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, BLOCK))
    top = torch.where(blocks.isfinite(), blocks.abs(), 0.0).amax(-1)
    man, exp = torch.frexp(top)  # top = man * 2^exp, man in [0.5, 1); 448 = 0.875 * 2^9
    exp = torch.where(man > F8_MAX / 512, exp - 8, exp - 9).clamp(min=-127)
    exp = torch.where(top == 0, 0, exp)
    codes = torch.ldexp(torch.where(blocks.isfinite(), blocks, math.nan), -exp[..., None])
    codes = codes.to(torch.float8_e4m3fn).flatten(-2)[..., : x.shape[-1]]
    return codes, (exp + 127).to(torch.uint8)


def _plain_restore(codes, scales):
    s = torch.repeat_interleave(scales.int() - 127, BLOCK, dim=-1)[..., : codes.shape[-1]]
    return torch.ldexp(codes.float(), s)


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "rope":
        return _plain_rope(case, state)
    if case["op"] in ("save", "restore"):
        codes, scales = _plain_save(state["x"])
        if case["op"] == "save":
            return {"codes": codes, "scales": scales}
        return {"x": _plain_restore(codes, scales).to(_dtype(case))}
    return _plain_attention(case, state)


def _own(case, st):
    from mla_attention_sequence_gb300 import laga
    if case["op"] == "rope":
        q, k = laga.rope(st["q"], st["k_rope"], st["pos"], sections=st["sections"], theta=case["theta"],
                         interleaved=case["interleaved"], inverse=case["inverse"])
        return {"q": q, "k_rope": k}
    if case["op"] == "save":
        p = laga.pack8(st["x"])
        return {"codes": p.codes.view(torch.float8_e4m3fn), "scales": p.scales}
    if case["op"] == "restore":
        return {"x": laga.unpack8(laga.pack8(st["x"]))}
    lo, hi = laga.key_bounds(st["doc_starts"], case["Sq"], q_offset=case["q_offset"], prefix=st["prefix"],
                             window=case["window"])
    mods = dict(key_lo=lo, key_hi=hi, softcap=case["softcap"], slopes=st["slopes"], q_offset=case["q_offset"],
                causal=not case["prefix"])
    x = (st["c_kv"], st["k_rope"], st["W_UK"], st["W_UV"])
    if case["op"] == "packed_bwd":
        q = laga.Packed8(st["q8"].contiguous().view(torch.uint8), st["q8_scales"], _dtype(case))
        out = laga.Packed8(st["out8"].contiguous().view(torch.uint8), st["out8_scales"], _dtype(case))
        return laga.masked_bwd(q, *x, out, st["lse"], st["dout"], **mods)
    if case["op"] == "fwd":
        return {"out": laga.masked_fwd(st["q"], *x, **mods)[0]}
    ws = laga.masked_workspace(st["q"], *x, **mods)
    out, lse = laga.masked_fwd(st["q"], *x, **mods, workspace=ws)
    return {"out": out, **laga.masked_bwd(st["q"], *x, out, lse, st["dout"], **mods, workspace=ws, reuse_kv=True)}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("save", "restore"):
        n = case["rows"] * case["cols"]
        packed = n + case["rows"] * (-(-case["cols"] // BLOCK))
        # restore: the checkpoint is written by one call and read by the next
        return {"bytes": n * e + packed if case["op"] == "save" else 2 * n * e + 2 * packed, "flops": 3 * n}
    if case["op"] == "rope":
        rows = case["B"] * case["S"]
        n = rows * (case["n_h"] * (case["d_nope"] + case["d_rope"]) + case["d_rope"])
        return {"bytes": 2 * n * e + 4 * case["axes"] * rows, "flops": 3 * rows * (case["n_h"] + 1) * case["d_rope"]}
    lo, hi = _bounds_np(case)
    B, Sq, S, n_h = case["B"], case["Sq"], case["S"], case["n_h"]
    pairs = int(np.maximum(hi - lo, 0).sum())
    seen = 0
    for b in range(B):  # keys that some row sees
        edge = np.zeros(S + 1, np.int64)
        some = hi[b] > lo[b]
        np.add.at(edge, lo[b][some], 1)
        np.add.at(edge, hi[b][some], -1)
        seen += int((np.cumsum(edge)[:S] > 0).sum())
    dqk, dv = case["d_nope"] + case["d_rope"], case["d_v"]
    weights = case["d_c"] * n_h * (case["d_nope"] + dv)
    q, out, lat = B * Sq * n_h * dqk, B * Sq * n_h * dv, B * S * (case["d_c"] + case["d_rope"])
    flops = 2 * pairs * n_h * (dqk + dv) + 2 * seen * weights
    if case["op"] == "fwd":
        # the latent rows that some row sees, read once
        return {"bytes": e * (q + out + seen * (case["d_c"] + case["d_rope"]) + weights), "flops": flops}
    if case["op"] == "packed_bwd":
        # q and out as codes and scales, dout; the gradients. K and V are rebuilt: once the forward's rebuild,
        # twice the forward's whole
        packed = q + out + B * Sq * n_h * (-(-dqk // BLOCK) + -(-dv // BLOCK))
        return {"bytes": packed + e * (q + out + 2 * lat + 2 * weights) + 4 * B * Sq * n_h,
                "flops": 2 * flops + 2 * seen * weights}
    return {"bytes": e * (2 * q + 2 * out + 2 * lat + 2 * weights), "flops": 3 * flops}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("save", "restore"):
        codes, _, back = _exact_codes(st["x"].double())
        return {"codes": codes, "scales": None} if case["op"] == "save" else {"x": back}
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["B"] * case["n_h"] * case["Sq"] * case["S"] > 1.2e9:
        return None
    return _exact_attention(case, st)


def _exact_codes(x):
    """Block by block in 64 bits: (values of the codes, scale exponents, values they stand for)."""
    codes, back, exps = torch.empty_like(x), torch.empty_like(x), []
    for k in range(0, x.shape[-1], BLOCK):
        blk = x[..., k:k + BLOCK]
        top = blk.abs().amax(-1, keepdim=True)
        e = torch.where(top > 0, torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / F8_MAX)), 0.0).clamp(min=-127)
        y = blk / torch.exp2(e)
        # e4m3: three fraction bits down to 2^-6, then steps of 2^-9; ties to even
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
        y = torch.round(y / step) * step
        codes[..., k:k + BLOCK], back[..., k:k + BLOCK] = y, y * torch.exp2(e)
        exps.append(e)
    return codes, torch.cat(exps, -1), back


def _exact_rope(case, st):
    n, dn = case["d_rope"] // 2, case["d_nope"]
    pos = st["pos"].cpu().numpy().astype(np.float64)
    axis = np.concatenate([np.full(s, a) for a, s in enumerate(st["sections"])])
    ang = np.stack([pos[axis[i]] * case["theta"] ** (-i / n) for i in range(n)], -1)  # [B, S, n]
    turn = np.exp(1j * (-ang if case["inverse"] else ang))

    def rotate(x, turn):
        z = x[..., 0::2] + 1j * x[..., 1::2] if case["interleaved"] else x[..., :n] + 1j * x[..., n:]
        z = z * turn
        y = np.empty_like(x)
        if case["interleaved"]:
            y[..., 0::2], y[..., 1::2] = z.real, z.imag
        else:
            y[..., :n], y[..., n:] = z.real, z.imag
        return y

    q, k = st["q"].double().cpu().numpy(), st["k_rope"].double().cpu().numpy()
    return {"q": np.concatenate([q[..., :dn], rotate(q[..., dn:], turn[:, :, None])], -1), "k_rope": rotate(k, turn)}


def _exact_attention(case, st):
    packed = case["op"] == "packed_bwd"
    x = {k: st[k].double().requires_grad_(True) for k in ("c_kv", "k_rope", "W_UK", "W_UV")}
    decode = lambda k: st[k].double() * torch.exp2(  # noqa: E731
        st[k + "_scales"].double() - 127).repeat_interleave(BLOCK, -1)[..., :st[k].shape[-1]]
    q = (decode("q8") if packed else st["q"].double()).requires_grad_(True)
    lo, hi = (torch.from_numpy(v).to(q.device) for v in _bounds_np(case))
    B, S, Sq, n_h = case["B"], case["S"], case["Sq"], case["n_h"]
    key = torch.arange(S, device=lo.device)
    pos = case["q_offset"] + torch.arange(Sq, device=lo.device)
    hidden = ((key < lo[..., None]) | (key >= hi[..., None]))[:, None]  # [B, 1, Sq, S]
    with torch.set_grad_enabled(case["op"] != "fwd"):
        K = torch.einsum("bsc,chd->bshd", x["c_kv"], x["W_UK"].view(case["d_c"], n_h, case["d_nope"]))
        V = torch.einsum("bsc,chd->bshd", x["c_kv"], x["W_UV"].view(case["d_c"], n_h, case["d_v"]))
        s = torch.einsum("bihd,bjhd->bhij", q[..., :case["d_nope"]], K)
        s = s + torch.einsum("bihd,bjd->bhij", q[..., case["d_nope"]:], x["k_rope"])
        s = s / math.sqrt(case["d_nope"] + case["d_rope"])
        if case["softcap"]:
            s = case["softcap"] * torch.tanh(s / case["softcap"])
        if st["slopes"] is not None:
            s = s - st["slopes"].double()[:, None, None] * (pos[:, None] - key).abs()
        s = s.masked_fill(hidden, -1e300)
        lse = st["lse"].double()[..., None] if packed else torch.logsumexp(s, -1, keepdim=True)
        P = torch.exp(s - torch.where(lse < -1e30, 0.0, lse)).masked_fill(hidden, 0.0)
        out = torch.einsum("bhij,bjhd->bihd", P, V)
        if case["op"] == "fwd":
            return {"out": out}
        dout = st["dout"].double()
        loss = (dout * out).sum()
        if packed:
            # the saved lse is a constant here, and D = rowsum(dout out) comes from the restored out: the
            # gradient of <dout, out> - <D, row sums of P> is P (dout V - D) in every score
            loss = loss - ((dout * decode("out8")).sum(-1).transpose(1, 2)[..., None] * P).sum()
        loss.backward()
    g = {"dq": q.grad, "dc_kv": x["c_kv"].grad, "dk_rope": x["k_rope"].grad, "dW_UK": x["W_UK"].grad,
         "dW_UV": x["W_UV"].grad}
    return g if packed else {"out": out.detach(), **g}
