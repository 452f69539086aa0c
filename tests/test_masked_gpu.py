"""The packed-document operators on the GPU against their definitions in 64 bits.

Tolerances (2-norm of the error over the 2-norm of the result, or of its uncancelled size where
the exact result cancels): a bf16 rounding is off by at most 2^-8 of the value, 2^-8 / sqrt(3) =
2.3e-3 in the root mean square. A bf16 output carries at most four independent ones (the rebuilt K
through the score, V, P, the result), a gradient six (those, dS, the stored dK or dV): sqrt(6) *
2.3e-3 = 5.6e-3, doubled for scores above 1 (K's rounding acts on the weight in proportion to the
score). fp32: 2^-24 per operation, sums of a few hundred terms and a handful of chained products,
exp and tanh of a few ulp: 100 * 2^-24 = 6e-6, doubled."""
import math

import numpy as np
import pytest
import torch

import masked_reference as ref
from mla_attention_sequence_gb300 import build, laga

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 1.2e-2, torch.float32: 1.2e-5}
DSV3 = (512, 128, 64, 128)
GRADS = ("dq", "dc_kv", "dk_rope", "dW_UK", "dW_UV")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def dev():
    return torch.device("cuda", 0)


def inputs(B, Sq, S, n_h, dims, dtype, seed=0):
    d_c, dn, dr, dv = dims
    g = torch.Generator(device=dev()).manual_seed(seed)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device=dev()) * std).to(dtype)
    x = dict(q=normal(B, Sq, n_h, dn + dr), c_kv=normal(B, S, d_c), k_rope=normal(B, S, dr),
             W_UK=normal(d_c, n_h * dn, std=d_c ** -0.5), W_UV=normal(d_c, n_h * dv, std=d_c ** -0.5))
    return x, normal(B, Sq, n_h, dv)


def step(x, dout, variant="auto", **kw):
    ws = laga.masked_workspace(*x.values(), variant=variant, **kw).fill_(255)  # NaN wherever it is not written
    out, lse = laga.masked_fwd(*x.values(), variant=variant, workspace=ws, **kw)
    g = laga.masked_bwd(*x.values(), out, lse, dout, variant=variant, workspace=ws, reuse_kv=True, **kw)
    return {"out": out, "lse": lse, **g}


def check(x, dout, tol=None, variant="auto", **kw):
    B, Sq = x["q"].shape[:2]
    S = x["c_kv"].shape[1]
    geo = {k: kw[k] for k in ("q_offset", "q_split", "q_offset2") if k in kw}
    seen = ref.visible(Sq, S, kw.get("key_lo"), kw.get("key_hi"), kw.get("causal", True), B=B, **geo)
    want = ref.attention(x, seen, kw.get("softcap", 0.0), kw.get("slopes"), kw.get("softmax_scale"),
                         ref.positions(Sq, kw.get("q_offset", 0), kw.get("q_split", 0), kw.get("q_offset2", 0)), dout)
    got = step(x, dout, variant, **kw)
    laga.check(dev())
    tol = tol or TOL[x["q"].dtype]
    ref.close(got, want, tol, ("out", *GRADS))
    # lse: an absolute error, of the scores' size (K's rounding) in bf16; in fp32 half a step of the lse
    # itself is 2^-24 of it (2.7e-5 at the 450 of the large scores' test, so an error no wider than 2e-5
    # cannot be met there), and the score behind it has a product, a scale and a bias of that size: 8 steps
    e = want["lse"] == -math.inf
    assert torch.equal(got["lse"] == -math.inf, e.to(dev()))
    err = (got["lse"].double() - want["lse"])[~e].abs()
    bound = 5e-2 if x["q"].dtype == torch.bfloat16 else 2e-5 + 8 * 2.0 ** -24 * want["lse"][~e].abs()
    assert bool((err <= bound).all())
    empty = ~seen.any(-1).to(dev())
    assert not got["out"][empty].any() and not got["dq"][empty].any()
    return got


def slopes(n_h):
    return torch.tensor([2.0 ** (-4.0 * (h + 1) / n_h) for h in range(n_h)], device=dev())


def random_bounds(B, Sq, S, seed, empty=0.2):
    """Any intervals: not monotone, some empty, some past the ends (which are clamped)."""
    g = torch.Generator().manual_seed(seed)
    lo = torch.randint(-5, S, (B, Sq), generator=g)
    hi = lo + torch.randint(1, S + 9, (B, Sq), generator=g)
    hi = torch.where(torch.rand(B, Sq, generator=g) < empty, lo - torch.randint(0, 3, (B, Sq), generator=g), hi)
    return lo.int().to(dev()), hi.int().to(dev())


MODS = {"mask": {}, "cap": dict(softcap=3.0), "bias": dict(slopes=True), "both": dict(softcap=8.0, slopes=True)}
SHAPES = {  # B, Sq, S, n_h
    "one": (1, 1, 1, 1), "token": (1, 1, 130, 2), "row": (2, 3, 129, 1), "tile": (1, 128, 128, 3),
    "ragged": (2, 200, 333, 3), "heads4": (1, 321, 700, 4), "wide": (1, 130, 1500, 2)}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("mod", MODS)
def test_any_intervals_bf16(shape, mod):
    B, Sq, S, n_h = SHAPES[shape]
    x, dout = inputs(B, Sq, S, n_h, DSV3, torch.bfloat16, 1)
    kw = dict(MODS[mod])
    if "slopes" in kw:
        kw["slopes"] = slopes(n_h)
    lo, hi = random_bounds(B, Sq, S, 7, empty=0.0 if Sq == 1 else 0.2)
    check(x, dout, key_lo=lo, key_hi=hi, causal=False, q_offset=S // 3, **kw)


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("shape,dims", [
    ((1, 1, 1, 1), (1, 1, 0, 1)), ((1, 1, 40, 2), (8, 5, 2, 3)), ((2, 65, 65, 3), (64, 32, 16, 32)),
    ((1, 100, 171, 2), (20, 40, 24, 56)), ((1, 70, 90, 2), (24, 100, 28, 120)), ((1, 33, 70, 1), (40, 200, 56, 256))])
def test_any_intervals_f32(shape, dims, mod):
    B, Sq, S, n_h = shape
    x, dout = inputs(B, Sq, S, n_h, dims, torch.float32, 2)
    kw = dict(MODS[mod])
    if "slopes" in kw:
        kw["slopes"] = slopes(n_h)
    lo, hi = random_bounds(B, Sq, S, 5, empty=0.0 if Sq == 1 else 0.2)
    check(x, dout, key_lo=lo, key_hi=hi, causal=False, q_offset=S // 3, **kw)


def test_bf16_on_the_cuda_cores():
    x, dout = inputs(1, 77, 150, 2, (48, 40, 8, 24), torch.bfloat16, 3)
    lo, hi = random_bounds(1, 77, 150, 6)
    check(x, dout, key_lo=lo, key_hi=hi, causal=False, softcap=5.0)
    x, dout = inputs(1, 40, 150, 2, DSV3, torch.bfloat16, 3)
    check(x, dout, variant="simt", q_offset=110, slopes=slopes(2))


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
@pytest.mark.parametrize("window,prefix", [(0, False), (50, False), (0, True)])
def test_packed_documents(dtype, dims, window, prefix):
    B, S = 2, 500
    starts = [[0, 1, 130, 130, 400, 460], [3, 60, 256, 384, 499, 500]]
    pre = [[1, 20, 5, 300, 0], [100, 30, 0, 7, 1]] if prefix else None
    Sq, off = 372, 128
    x, dout = inputs(B, Sq, S, 2, dims, dtype, 4)
    st = torch.tensor(starts, dtype=torch.int32, device=dev())
    pt = torch.tensor(pre, dtype=torch.int32, device=dev()) if prefix else None
    lo, hi = laga.key_bounds(st, Sq, q_offset=off, prefix=pt, window=window)
    want = ref.bounds(starts, Sq, S, off, pre, window)
    assert torch.equal(lo.cpu().long(), torch.from_numpy(want[0])) and torch.equal(hi.cpu().long(),
                                                                                   torch.from_numpy(want[1]))
    check(x, dout, key_lo=lo, key_hi=hi, q_offset=off, causal=not prefix, softcap=6.0, slopes=slopes(2))


def test_key_bounds_two_segments_and_outside():
    starts = [[5, 9, 9, 300, 700]]
    st = torch.tensor(starts, dtype=torch.int32, device=dev())
    lo, hi = laga.key_bounds(st, 256, q_offset=0, q_split=128, q_offset2=640, skv=650, window=7)
    want = ref.bounds(starts, 256, 650, 0, None, 7, 128, 640)
    # past skv the upper bound is clamped; the interval may be empty then
    assert torch.equal(lo.cpu().long(), torch.from_numpy(want[0])) and torch.equal(hi.cpu().long(),
                                                                                   torch.from_numpy(want[1]))


@pytest.mark.parametrize("mod", ["mask", "both"])
def test_most_key_tiles_unseen(mod):
    """A few short intervals far apart: the other key tiles are neither rebuilt nor given gradients."""
    B, Sq, S, n_h = 3, 190, 9000, 2
    x, dout = inputs(B, Sq, S, n_h, DSV3, torch.bfloat16, 14)
    g = torch.Generator().manual_seed(3)
    at = torch.tensor([[0, 5000], [8990, 3], [200, 330]])[:, :, None].expand(B, 2, 95).reshape(B, Sq)
    lo = (at + torch.randint(0, 20, (B, Sq), generator=g)).int()
    hi = (lo + torch.randint(1, 90, (B, Sq), generator=g)).int()
    kw = dict(MODS[mod], key_lo=lo.to(dev()), key_hi=hi.to(dev()), causal=False, q_offset=4000)
    if mod == "both":
        kw["slopes"] = slopes(n_h) / 64
    got = check(x, dout, **kw)
    seen = ref.visible(Sq, S, lo, hi, causal=False, B=B).any(1).to(dev())
    assert not got["dc_kv"][~seen].any() and not got["dk_rope"][~seen].any()


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("docs", ["one", "many", "uneven"])
def test_many_tiles_per_sm(docs, mod):
    """Several (head, query tile) items and CTAs of each kernel on every SM, walks of one to eleven key tiles."""
    B, S, n_h = 2, 1300, 24
    starts = {"one": [[0, 1300], [7, 1290]], "uneven": [[0, 3, 900, 910, 1300], [0, 600, 601, 1000, 1000]],
              "many": [list(range(0, 1300, 43))[:31], list(range(5, 1300, 42))[:31]]}[docs]
    x, dout = inputs(B, S, S, n_h, DSV3, torch.bfloat16, 24)
    kw = dict(MODS[mod])
    if "slopes" in kw:
        kw["slopes"] = slopes(n_h)
    lo, hi = laga.key_bounds(torch.tensor(starts, dtype=torch.int32, device=dev()), S)
    check(x, dout, key_lo=lo, key_hi=hi, **kw)


def test_long_rows_without_mods():
    """The form for walks that can be long, with several query tiles and heads, and rows that see little."""
    B, Sq, S, n_h = 1, 400, 8300, 6
    x, dout = inputs(B, Sq, S, n_h, DSV3, torch.bfloat16, 25)
    lo, hi = random_bounds(B, Sq, S, 8)
    check(x, dout, key_lo=lo, key_hi=hi, causal=False, q_offset=7000)


def test_two_segments():
    B, Sq, S, n_h = 1, 256 + 70, 1024, 4
    x, dout = inputs(B, Sq, S, n_h, DSV3, torch.bfloat16, 5)
    geo = dict(q_offset=100, q_split=256, q_offset2=900)
    st = torch.tensor([[0, 150, 333, 880, 960, 1024]], dtype=torch.int32, device=dev())
    lo, hi = laga.key_bounds(st, Sq, **geo)
    check(x, dout, key_lo=lo, key_hi=hi, slopes=slopes(n_h), **geo)


def test_without_mods_is_the_plain_attention():
    """No bounds, no cap, no bias: laga.fwd / bwd's results (a row's running maximum may differ, and with
    it the rounding of its weights), the backward's to the bit on the same out and lse."""
    x, dout = inputs(2, 300, 700, 4, DSV3, torch.bfloat16, 6)
    got = check(x, dout, q_offset=400)
    g = laga.bwd(*x.values(), got["out"], got["lse"], dout, q_offset=400)
    for k in set(GRADS) - {"dk_rope"}:
        assert torch.equal(got[k], g[k]), k
    # the heads of dk_rope are summed in fp32 in other groups: 2^-22 of the summands, then one rounding to
    # bf16 that may fall on the other side (a step, 2^-7)
    a, b = got["dk_rope"].float(), g["dk_rope"].float()
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -20 * b.abs().max()).all())
    again = step(x, dout, q_offset=400)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_non_finite_values_in_masked_places(dtype, dims, value):
    B, Sq, S, n_h = 2, 260, 260, 2
    starts = [[0, 100, 230], [0, 31, 251]]  # the rest is padding
    st = torch.tensor(starts, dtype=torch.int32, device=dev())
    lo, hi = laga.key_bounds(st, Sq)
    x, dout = inputs(B, Sq, S, n_h, dims, dtype, 7)
    kw = dict(key_lo=lo, key_hi=hi, softcap=9.0)
    clean = step(x, dout, **kw)
    y, dy = {k: v.clone() for k, v in x.items()}, dout.clone()
    for b, end in ((0, 230), (1, 251)):
        y["c_kv"][b, end:, ::3] = value
        y["k_rope"][b, end + 1:, 0] = value
        y["q"][b, end:] = value
        dy[b, end:, :, 1] = value
    got = step(y, dy, **kw)
    for k in clean:
        assert torch.equal(got[k], clean[k]), k
    # a key of the second document of batch element 0: its document from it on, nothing else
    y = {k: v.clone() for k, v in x.items()}
    y["c_kv"][0, 150, 5] = value
    got = step(y, dout, **kw)
    hit = torch.zeros(B, Sq, dtype=torch.bool, device=dev())
    hit[0, 150:230] = True
    assert got["out"][hit].isnan().all() and torch.equal(got["out"][~hit], clean["out"][~hit])
    assert got["dq"][hit].isnan().all() and torch.equal(got["dq"][~hit], clean["dq"][~hit])
    keys = torch.zeros(B, S, dtype=torch.bool, device=dev())
    keys[0, 100:230] = True  # seen by a row that is hit
    assert got["dc_kv"][keys].isnan().all() and torch.equal(got["dc_kv"][~keys], clean["dc_kv"][~keys])
    assert got["dk_rope"][keys].isnan().all() and torch.equal(got["dk_rope"][~keys], clean["dk_rope"][~keys])
    # a query row of the same document: itself and the keys that it sees
    for name in ("q", "dout"):
        y, dy = {k: v.clone() for k, v in x.items()}, dout.clone()
        (y["q"] if name == "q" else dy)[0, 180, 1, 3] = value
        got = step(y, dy, **kw)
        keys[:] = False
        keys[0, 100:181] = True
        assert got["dc_kv"][keys].isnan().all() and torch.equal(got["dc_kv"][~keys], clean["dc_kv"][~keys])
        row = torch.zeros(B, Sq, n_h, dtype=torch.bool, device=dev())
        row[0, 180, 1] = True
        assert got["dq"][row].isnan().all() and torch.equal(got["dq"][~row], clean["dq"][~row])


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
@pytest.mark.parametrize("softcap,bias", [(1e-20, False), (600.0, False), (2e4, True), (1e30, False)])
def test_caps_from_one_end_of_their_range_to_the_other(dtype, dims, softcap, bias):
    """The smallest makes every visible key weigh the same (and no score a gradient), the largest does
    nothing; tanh of a score far below its cap has to be right relative to the score."""
    x, dout = inputs(1, 140, 140, 2, dims, dtype, 8)
    lo, hi = random_bounds(1, 140, 140, 3)
    check(x, dout, key_lo=lo, key_hi=hi, softcap=softcap, slopes=slopes(2) if bias else None)


@pytest.mark.parametrize("dtype,dims,S", [(torch.bfloat16, DSV3, 130), (torch.bfloat16, DSV3, 8192),
                                          (torch.float32, (32, 16, 8, 24), 130)])
def test_scores_that_are_all_minus_infinity(dtype, dims, S):
    """A row that sees one key, with an infinite q whose product with it is -inf: exp(-inf + inf), a NaN,
    and not the zero of a row that sees nothing."""
    x, dout = inputs(1, 130, S, 2, dims, dtype, 9)
    x["k_rope"][0, 0, 0] = -1.0
    clean = step(x, dout)
    y = {k: v.clone() for k, v in x.items()}
    y["q"][0, 0, 1, dims[1]] = math.inf
    got = step(y, dout)
    row = torch.zeros(1, 130, 2, dtype=torch.bool, device=dev())
    row[0, 0, 1] = True
    for k in ("out", "dq"):
        assert got[k][row].isnan().all() and torch.equal(got[k][~row], clean[k][~row]), k
    assert got["lse"][0, 1, 0].isnan() and got["lse"].isnan().sum() == 1
    for k in ("dc_kv", "dk_rope"):
        assert got[k][0, 0].isnan().all() and torch.equal(got[k][0, 1:], clean[k][0, 1:]), k


def test_large_scores_and_far_bias():
    """Scores of a few hundred, a bias that leaves one key: the weights stay those of the definition."""
    x, dout = inputs(1, 150, 300, 2, (16, 8, 4, 8), torch.float32, 8)
    x["q"] = x["q"] * 60
    # K's fp32 rounding acts on the weights times the score's size (up to ~500)
    check(x, dout, tol=500 * TOL[torch.float32], q_offset=150, slopes=torch.tensor([30.0, -1.5], device=dev()))


def test_gradients_by_differences_f32():
    """Directional differences of the fp32 forward: h = 2^-6 leaves h^2 / 6 of the third derivative
    (4e-5 of it) and the forward's rounding, 2^-24 * sqrt(values) / h: 5e-3 covers both."""
    x, dout = inputs(1, 90, 120, 2, (24, 16, 8, 16), torch.float32, 9)
    st = torch.tensor([[0, 45, 118]], dtype=torch.int32, device=dev())
    lo, hi = laga.key_bounds(st, 90, q_offset=30)
    kw = dict(key_lo=lo, key_hi=hi, q_offset=30, softcap=2.0, slopes=slopes(2))
    g = step(x, dout, **kw)
    for k, name in zip(x, ("dq", "dc_kv", "dk_rope", "dW_UK", "dW_UV")):
        d = torch.randn_like(x[k])
        d = d / d.norm() * x[k].norm() * 0.5
        h = 2.0 ** -6
        f = [float((laga.masked_fwd(*{**x, k: x[k] + s * h * d}.values(), **kw)[0].double() * dout.double()).sum())
             for s in (1, -1)]
        num, want = (f[0] - f[1]) / (2 * h), float((g[name].double() * d.double()).sum())
        size = float(g[name].double().norm() * d.double().norm())
        assert abs(num - want) <= 5e-3 * size, (name, num, want, size)


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 40, 12, 70))])
def test_backward_from_checkpoints(dtype, dims):
    B, Sq, S, n_h = 2, 150, 290, 2
    x, dout = inputs(B, Sq, S, n_h, dims, dtype, 10)
    lo, hi = random_bounds(B, Sq, S, 11)
    kw = dict(key_lo=lo, key_hi=hi, causal=False, softcap=4.0)
    out, lse = laga.masked_fwd(*x.values(), **kw)
    q8, out8 = laga.pack8(x["q"]), laga.pack8(out)
    rest = list(x.values())[1:]
    got = laga.masked_bwd(q8, *rest, out8, lse, dout, **kw)
    # the same backward on the restored tensors, to the bit
    same = laga.masked_bwd(laga.unpack8(q8), *rest, laga.unpack8(out8), lse, dout, **kw)
    for k in GRADS:
        assert torch.equal(got[k], same[k]), k
    seen = ref.visible(Sq, S, lo, hi, causal=False, B=B)
    want = ref.attention({**x, "q": laga.unpack8(q8)}, seen, 4.0, None, None, None, dout, lse=lse,
                         out=laga.unpack8(out8))
    ref.close(got, want, TOL[dtype], GRADS)


# ---------------------------------------------------------------- rotation

def rope_reference(x, pos, sections, theta, interleaved, inverse):
    """x [B, S, .., d] in complex128."""
    x = x.double().cpu().numpy()
    n = x.shape[-1] // 2
    axis = np.concatenate([np.full(s, a, np.int64) for a, s in enumerate(sections)])
    p = pos.cpu().numpy()[axis].astype(np.float64)  # [n, B, S]
    ang = np.moveaxis(p, 0, -1) * theta ** (-np.arange(n) / n)
    turn = np.exp(1j * (-ang if inverse else ang)).reshape(x.shape[:2] + (1,) * (x.ndim - 3) + (n,))
    z = (x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :n] + 1j * x[..., n:]) * turn
    y = np.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:] = z.real, z.imag
    return torch.from_numpy(y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,S,n_h,dn,dr,sections", [
    (1, 1, 1, 0, 2, [1]), (2, 5, 3, 128, 64, [8, 12, 12]), (1, 300, 16, 128, 64, [32]), (2, 7, 2, 3, 10, [2, 0, 3]),
    (1, 33, 5, 40, 24, [6, 6]), (1, 9, 2, 12, 256, [1, 2, 3, 122])])
def test_rope(dtype, interleaved, B, S, n_h, dn, dr, sections):
    g = torch.Generator(device=dev()).manual_seed(1)
    q = torch.randn(B, S, n_h, dn + dr, generator=g, device=dev()).to(dtype)
    k = torch.randn(B, S, dr, generator=g, device=dev()).to(dtype)
    pos = torch.randint(-3000, 2000000, (len(sections), B, S), generator=g, device=dev(), dtype=torch.int32)
    # one rounding to the type, and 2^-24 of the sine, the cosine, the two products and their sum
    tol = 2.0 ** -8 if dtype == torch.bfloat16 else 8 * 2.0 ** -24
    for inverse in (False, True):
        a, b = laga.rope(q, k, pos, sections, 1e4, interleaved, inverse)
        assert torch.equal(a[..., :dn], q[..., :dn])
        for got, src in ((a[..., dn:], q[..., dn:]), (b, k)):
            want = rope_reference(src, pos, sections, 1e4, interleaved, inverse)
            size = max(1.0, float(src.abs().max())) * 2 ** 0.5
            assert float((got.double().cpu() - want).abs().max()) <= tol * size
    a64, b64 = laga.rope(q, k, pos.long(), sections, 1e4, interleaved, True)
    assert torch.equal(a, a64) and torch.equal(b, b64)
    qi, ki = q.clone(), k.clone()
    r = laga.rope(qi, ki, pos, sections, 1e4, interleaved, True, q_out=qi, k_out=ki)
    assert r[0] is qi and torch.equal(qi, a) and torch.equal(ki, b)


def test_rope_far_positions_and_gradient():
    """Positions of 2^40 turn exactly as their remainder does; the inverse is the transpose."""
    g = torch.Generator(device=dev()).manual_seed(2)
    q = torch.randn(1, 6, 2, 24, generator=g, device=dev())
    k = torch.randn(1, 6, 8, generator=g, device=dev())
    pos = torch.tensor([[[2 ** 40 + 3, -2 ** 33, 2 ** 31, 0, 1, -1]]], device=dev())
    a, b = laga.rope(q, k, pos, theta=100.0)
    # the reference's double product is off by 2^40 * 2^-53 = 1.2e-4 rad there
    want = rope_reference(k, pos, [4], 100.0, True, False)
    assert float((b.double().cpu() - want).abs().max()) <= 4e-4 * float(k.abs().max())
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    gq, gk = laga.rope(dq, dk, pos, theta=100.0, inverse=True)
    for u, v, w, z in ((a, dq, q, gq), (b, dk, k, gk)):  # <R x, d> = <x, R^T d>
        lhs, rhs = float((u.double() * v.double()).sum()), float((w.double() * z.double()).sum())
        assert abs(lhs - rhs) <= 16 * 2.0 ** -24 * float(u.norm() * v.norm())


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 192), (9, 77), (130, 64), (1, 513)])
def test_checkpoints(dtype, rows, cols):
    g = torch.Generator(device=dev()).manual_seed(rows * cols)
    size = torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=dev()).float())
    x = (torch.randn(rows, cols, generator=g, device=dev()) * size *
         torch.exp2(torch.randint(-18, 1, (rows, cols), generator=g, device=dev()).float())).to(dtype)
    x[0, 0] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2, :40] = torch.tensor([math.inf, -math.inf, math.nan, 448.0, 449.0, 1e-38, -1e-40, 3e38] * 5,
                                 device=dev())[:min(cols, 40)].to(dtype)
    check_checkpoint(x)


def check_checkpoint(x):
    rows, cols = x.shape
    p = laga.pack8(x)
    vals, scales = ref.pack8(x.double().cpu().numpy())
    assert p.scales.shape == scales.shape and torch.equal(p.scales.cpu().long(), torch.from_numpy(scales))
    got = torch.from_numpy(ref.e4m3_values()[p.codes.cpu().numpy()])
    np.testing.assert_array_equal(got.numpy(), vals)
    back = laga.unpack8(p)
    want = torch.from_numpy(vals * np.exp2(np.repeat(scales - 127.0, 32, 1)[:, :cols])).to(x.dtype)
    assert back.dtype == x.dtype and torch.equal(back.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_checkpoint_of_special_blocks():
    """Largest sizes at the scale's steps (448 * 2^k and just above), ties, the range's ends."""
    rows = []
    for top in (448.0, 448.0 * 2, 449.0, 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -149, 3.3e38, 2.0 ** 127):
        r = torch.linspace(-1, 1, 32) * top
        r[5] = top
        rows.append(r)
    ties = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 2 ** -10, 3 * 2 ** -10, 17.0, 19.0] * 4)
    x = torch.stack(rows + [ties]).to(dev())
    check_checkpoint(x)
    check_checkpoint(x.bfloat16())


def test_checkpoints_of_unaligned_and_empty_tensors():
    base = torch.randn(64 * 9 + 1, device=dev()).bfloat16()
    x = base[1:].view(9, 64)  # 2-byte aligned
    p, q = laga.pack8(x), laga.pack8(x.clone())
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    out = torch.empty(64 * 9 + 1, device=dev(), dtype=torch.bfloat16)[1:].view(9, 64)
    assert torch.equal(laga.unpack8(p, out), laga.unpack8(q))
    e = laga.pack8(torch.empty(0, 64, device=dev()))
    assert e.codes.shape == (0, 64) and laga.unpack8(e).shape == (0, 64)


# ---------------------------------------------------------------- as they are used

def chain(x, pos, st, sections, dout):
    """Rotate, attend, save q and out in 8 bits, back from the checkpoints, rotate back."""
    q, kr = laga.rope(x["q"], x["k_rope"], pos, sections)
    rest = (x["c_kv"], kr, x["W_UK"], x["W_UV"])
    lo, hi = laga.key_bounds(st, q.shape[1])
    kw = dict(key_lo=lo, key_hi=hi, softcap=20.0)
    out, lse = laga.masked_fwd(q, *rest, **kw)
    q8, out8 = laga.pack8(q), laga.pack8(out)
    g = laga.masked_bwd(q8, *rest, out8, lse, dout, **kw)
    dq, dkr = laga.rope(g["dq"], g["dk_rope"], pos, sections, inverse=True)
    return {"out": out, **g, "dq": dq, "dk_rope": dkr}


def chain_case(dtype=torch.bfloat16, dims=DSV3, seed=12):
    x, dout = inputs(2, 300, 300, 4, dims, dtype, seed)
    n = dims[2] // 2
    sections = [n // 2, n // 4, n - n // 2 - n // 4]
    pos = torch.randint(0, 5000, (3, 2, 300), device=dev(), dtype=torch.int32)
    st = torch.tensor([[0, 77, 290], [0, 128, 300]], dtype=torch.int32, device=dev())
    return x, pos, st, sections, dout


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
def test_chain(dtype, dims):
    """The whole chain against 64 bits, with the checkpoints' own error counted: half a step of e4m3
    (2^-4) in the root mean square over sqrt(3) on q and out moves each gradient by about as much."""
    x, pos, st, sections, dout = chain_case(dtype, dims)
    got = chain(x, pos, st, sections, dout)
    xr = {k: v.double() for k, v in x.items()}
    xr["q"] = torch.cat([xr["q"][..., :dims[1]],
                         rope_reference(x["q"][..., dims[1]:], pos, sections, 1e4, True, False).to(dev())], -1)
    xr["k_rope"] = rope_reference(x["k_rope"], pos, sections, 1e4, True, False).to(dev())
    lo, hi = ref.bounds(st.tolist(), 300, 300)
    seen = ref.visible(300, 300, torch.from_numpy(lo), torch.from_numpy(hi), B=2)
    want = ref.attention(xr, seen, 20.0, dout=dout)
    ref.close(got, want, TOL[dtype], ("out",))
    want["dk_rope"] = rope_reference(want["dk_rope"], pos, sections, 1e4, True, True)
    want["dq"] = torch.cat([want["dq"][..., :dims[1]].cpu(),
                            rope_reference(want["dq"][..., dims[1]:], pos, sections, 1e4, True, True)], -1)
    ref.close(got, want, 3 * 2.0 ** -4 / 3 ** 0.5, GRADS)


def test_chain_captured_in_a_graph_and_on_another_stream():
    case = chain_case()
    want = chain(*case)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain(*case)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(*case)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    # other values, other documents, the same graph
    x, pos, st, sections, dout = chain_case(seed=13)
    for a, b in zip(case[0].values(), x.values()):
        a.copy_(b)
    case[1].copy_(pos)
    case[2].copy_(torch.tensor([[0, 5, 200], [10, 11, 288]], dtype=torch.int32))
    case[4].copy_(dout)
    graph.replay()
    torch.cuda.synchronize()
    new = chain(x, pos, case[2], sections, dout)
    for k in new:
        assert torch.equal(got[k], new[k]), k
    laga.check(dev())


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
def test_captured_behind_copies_and_a_join_of_streams(dtype, dims):
    """The chain's first kernel behind a copy, behind another stream's work and behind a chain that shares
    its workspace; two such graphs replayed one after the other without a wait between them."""
    kw = dict(softcap=9.0, slopes=slopes(3))
    problems, graphs, results = [], [], []
    x0, dout0 = inputs(1, 300, 300, 3, dims, dtype, 41)
    ws = laga.masked_workspace(*x0.values(), **kw)
    for seed, starts in ((41, [0, 100, 290]), (42, [0, 33, 34, 300])):
        x, dout = inputs(1, 300, 300, 3, dims, dtype, seed)
        st = torch.tensor([starts], dtype=torch.int32, device=dev())
        problems.append((x, dout, st))

    def work(x, dout, st):
        y = {k: v.clone() for k, v in x.items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lo, hi = laga.key_bounds(st, 300)
            q8 = laga.pack8(y["q"])
        torch.cuda.current_stream().wait_stream(side)
        m = dict(kw, key_lo=lo, key_hi=hi, workspace=ws)
        out, lse = laga.masked_fwd(*y.values(), **m)
        g = laga.masked_bwd(*y.values(), out, lse, dout, reuse_kv=True, **m)
        h = laga.masked_bwd(q8, *list(y.values())[1:], laga.pack8(out), lse, dout, **m)
        return {"out": out, "lse": lse, **g, **{k + " packed": v for k, v in h.items()}}

    want = [work(*p) for p in problems]
    torch.cuda.synchronize()
    for p in problems:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(work(*p))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for got, w in zip(results, want):
        for k in w:
            assert torch.equal(got[k], w[k]), k
    laga.check(dev())


def test_two_calls_at_once():
    """Two streams, each with its own workspace, overlapping."""
    a, b = chain_case(seed=20), chain_case(seed=21)
    want = [chain(*a), chain(*b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                got[i] = chain(*c)
    torch.cuda.synchronize()
    for i in (0, 1):
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), k


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24))])
def test_new_values_at_the_same_addresses(dtype, dims):
    """Steps enqueued one after the other without a wait, their inputs replaced in place between them: each
    sees its own (kernels of a call start before the one before them has ended)."""
    n, S, n_h = 6, 700, 4
    problems = [inputs(2, S, S, n_h, dims, dtype, 50 + i) for i in range(n)]
    starts = [torch.tensor([[0, 100 * i + 1, 640], [5, 300, 690 - i]], dtype=torch.int32, device=dev()) for i in range(n)]
    x, dout, st = {k: v.clone() for k, v in problems[0][0].items()}, problems[0][1].clone(), starts[0].clone()
    ws = laga.masked_workspace(*x.values())
    results = {False: [], True: []}
    for wait in (True, False):
        for (y, dy), s in zip(problems, starts):
            for k, v in y.items():
                x[k].copy_(v)
            dout.copy_(dy)
            st.copy_(s)
            lo, hi = laga.key_bounds(st, S)
            if wait:
                torch.cuda.synchronize()
            kw = dict(key_lo=lo, key_hi=hi, softcap=20.0, workspace=ws)
            out, lse = laga.masked_fwd(*x.values(), **kw)
            if wait:
                torch.cuda.synchronize()
            g = laga.masked_bwd(*x.values(), out, lse, dout, reuse_kv=True, **kw)
            if wait:
                torch.cuda.synchronize()
            h = laga.masked_bwd(laga.pack8(x["q"]), *list(x.values())[1:], laga.pack8(out), lse, dout, **kw)
            if wait:
                torch.cuda.synchronize()
            results[wait].append([out, lse, *g.values(), *h.values()])
    torch.cuda.synchronize()
    for a, b in zip(results[False], results[True]):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    laga.check(dev())


@pytest.mark.parametrize("kind", ["contiguous", "zigzag"])
def test_sequence_parallel_ranks_of_packed_documents(kind):
    """Each rank's local step, one after the other: their rows make up the whole sequence's out and dq,
    their latent and weight gradients add up to its (each rounded to bf16 once more: 2^-8)."""
    from mla_attention_sequence_gb300 import sp
    B, S, n_h = 2, 1024, 4
    x, dout = inputs(B, S, S, n_h, DSV3, torch.bfloat16, 22)
    st = torch.tensor([[0, 100, 700, 1000], [10, 333, 512, 1024]], dtype=torch.int32, device=dev())
    fwd, bwd = sp.packed_document_ops(st, window=300, softcap=20.0, slopes=slopes(n_h))
    lo, hi = laga.key_bounds(st, S, window=300)
    want = check(x, dout, key_lo=lo, key_hi=hi, softcap=20.0, slopes=slopes(n_h))
    layout = sp.Layout(S, 4, kind)
    sums = {k: torch.zeros(want[k].shape, device=dev()) for k in GRADS[1:]}
    for r in range(4):
        rows = layout.rows(r).to(dev())
        a = layout.query_args(r)
        args = (x["q"][:, rows].contiguous(), *list(x.values())[1:])
        at = (a["q_offset"], True, a["q_split"], a["q_offset2"])
        out, lse = fwd(*args, *at)
        g = bwd(*args, out, lse, dout[:, rows].contiguous(), *at)
        for got, full in ((out, want["out"][:, rows]), (g["dq"], want["dq"][:, rows])):
            assert float((got.double() - full.double()).norm()) <= 2.0 ** -8 * float(full.double().norm())
        for k in sums:
            sums[k] += g[k].float()
    for k, v in sums.items():
        assert float((v.double() - want[k].double()).norm()) <= 3 * 2.0 ** -8 * float(want[k].double().norm()), k


def test_a_scale_held_in_a_tensor():
    """Its value counts at each call, not the object."""
    x, _ = inputs(1, 40, 40, 2, (16, 8, 4, 8), torch.float32)
    scale = torch.tensor(0.25)
    for value in (0.25, 1.5):
        scale.fill_(value)
        out, lse = laga.masked_fwd(*x.values(), softmax_scale=scale)
        want, want_lse = laga.masked_fwd(*x.values(), softmax_scale=value)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("which", ["rows", "heads"])
def test_rope_of_nothing(which):
    q = torch.empty(1, 0, 2, 8, device=dev()) if which == "rows" else torch.empty(0, 3, 2, 8, device=dev())
    k = torch.empty(q.shape[0], q.shape[1], 4, device=dev())
    a, b = laga.rope(q, k, torch.zeros(1, *q.shape[:2], dtype=torch.int32, device=dev()))
    assert a.shape == q.shape and b.shape == k.shape


def test_argument_checks():
    x, dout = inputs(1, 8, 8, 2, (16, 8, 4, 8), torch.float32)
    lo = torch.zeros(1, 8, dtype=torch.int32, device=dev())
    with pytest.raises(TypeError, match="key_lo"):
        laga.masked_fwd(*x.values(), key_lo=lo.long())
    with pytest.raises(ValueError, match="key_hi"):
        laga.masked_fwd(*x.values(), key_hi=lo[:, :4])
    with pytest.raises(ValueError, match="slopes"):
        laga.masked_fwd(*x.values(), slopes=torch.zeros(3, device=dev()))
    with pytest.raises(laga.LagaError, match="softcap"):
        laga.masked_fwd(*x.values(), softcap=-1.0)
    out, lse = laga.masked_fwd(*x.values())
    with pytest.raises(ValueError, match="dout"):
        laga.masked_bwd(*x.values(), out, lse, dout[:, :4])
    with pytest.raises(ValueError, match="workspace"):
        laga.masked_bwd(*x.values(), out, lse, dout, reuse_kv=True)
    with pytest.raises(ValueError, match="workspace too small"):
        laga.masked_fwd(*x.values(), workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError, match="section"):
        laga.rope(x["q"], x["k_rope"], lo[None], [1, 1])
    with pytest.raises(ValueError, match="pos"):
        laga.rope(x["q"], x["k_rope"], lo[None, :, :4])
    with pytest.raises(laga.LagaError, match="sections"):
        laga.rope(x["q"], x["k_rope"], lo[None], [1])
