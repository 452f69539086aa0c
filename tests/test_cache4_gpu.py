"""The paged 4-bit latent cache on the GPU: rows written and read against the format's definition, attention
against its own in 64 bits over the values that the cache's bytes stand for.

Tolerances. Latents: none, the format is exact. Keys: as the norms with rotation. Attention (2-norms): fp32 as
the masked attention's, 100 * 2^-24 doubled. bf16: three independent roundings to bf16 (the query in the latent
space, which acts on the weights in proportion to the score, the context, the result), each at most 2^-8,
2.3e-3 in the root mean square: 4e-3, doubled for scores above 1. lse: an absolute error, of the scores' size."""
import math

import numpy as np
import pytest
import torch

import cache4_reference as cref
import masked_reference as ref
from mla_attention_sequence_gb300 import build, laga

pytestmark = pytest.mark.gpu
TOL = {torch.bfloat16: 8e-3, torch.float32: 200 * 2.0 ** -24}
DSV3 = (512, 128, 64, 128)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def dev():
    return torch.device("cuda", 0)


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def pool(pages, page, d_c, d_rope, dtype, seed=0):
    """A cache whose unused places hold what does most harm: blocks that read as NaN, NaN keys."""
    c = laga.cache4(pages, page, d_c, d_rope, dtype, dev())
    c.codes.random_(0, 256, generator=gen(seed))
    c.scales.fill_(255)
    c.k_rope.fill_(float("nan"))
    return c


def tables(lengths, page, spare=2, seed=0):
    """Shuffled pages for each sequence, -1 past its end; (table, pages of the pool)."""
    need = [-(-int(n) // page) for n in lengths]
    ids = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(lengths), max(1, *need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t.to(dev()), sum(need) + spare


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def filled(lengths, page, dims, dtype, seed=0, std=1.0):
    """A cache holding random tokens of those lengths, written by the library (its own tests are below)."""
    d_c, _, dr, _ = dims
    table, n = tables(lengths, page, seed=seed)
    c = pool(n, page, d_c, dr, dtype, seed)
    most = max(1, *lengths)
    x = (torch.randn(len(lengths), most, d_c, generator=gen(seed), device=dev()) * std).to(dtype)
    k = torch.randn(len(lengths), most, dr, generator=gen(seed + 1), device=dev()).to(dtype)
    laga.cache4_append(c, x, k, table, torch.zeros(len(lengths), dtype=torch.int32, device=dev()), counts=i32(*lengths),
                       theta=None)
    return c, table


# ---------------------------------------------------------------- rows
def latents(rows, d_c, dtype, seed):
    """Blocks of very different size, ties between codes, zeros, negative zeros, values past either end."""
    x = torch.randn(rows, d_c, generator=gen(seed), device=dev())
    x *= torch.exp2(torch.randint(-22, 18, (rows, -(-d_c // 16)), generator=gen(seed + 1), device=dev()).float()
                    ).repeat_interleave(16, 1)[:, :d_c]
    grid = torch.tensor([0, .25, .5, .75, 1.25, 1.75, 2.5, 3.5, 5, 6], device=dev())
    ties = grid[torch.randint(0, 10, (rows, d_c), generator=gen(seed + 2), device=dev())]
    ties[:, 0::16] = 6.0
    ties *= torch.sign(torch.randn(rows, d_c, generator=gen(seed + 3), device=dev())) * 2.0 ** torch.randint(
        -14, 12, (rows, 1), generator=gen(seed + 4), device=dev())
    which = torch.randint(0, 4, (rows, 1), generator=gen(seed + 5), device=dev())
    x = torch.where(which == 0, ties, x)
    return torch.where((which == 1) & (torch.arange(d_c, device=dev()) < 16), -0.0, x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d_c,d_rope,page,B,S", [(512, 64, 64, 3, 21), (512, 64, 1, 2, 5), (64, 16, 16, 2, 40), (1, 0, 3, 1, 7),
                                                 (17, 2, 5, 2, 11), (100, 30, 7, 2, 9), (1024, 256, 2, 1, 4)])
def test_rows_written_and_read(d_c, d_rope, page, B, S, dtype):
    starts = torch.randint(0, 30, (B,), generator=torch.Generator().manual_seed(d_c))
    counts = torch.tensor([S - (3 * b) % S for b in range(B)])
    table, n = tables(starts + counts, page)
    cache = pool(n, page, d_c, d_rope, dtype)
    before = cache.codes.clone(), cache.scales.clone()
    x = latents(B * S, d_c, dtype, 3).view(B, S, d_c)
    k = torch.randn(B, S, d_rope, generator=gen(9), device=dev()).to(dtype)
    w = torch.randn(d_rope, generator=gen(10), device=dev()).to(dtype) if d_rope else None
    laga.cache4_append(cache, x, k, table, starts.int().to(dev()), counts=counts.int().to(dev()), k_weight=w, theta=1e4)
    laga.check(dev())
    codes, scales, vals = cref.encode(x.view(B * S, -1).double().cpu().numpy())
    want_codes, want_scales = (t.cpu().view(n * page, -1).clone() for t in before)
    touched = torch.zeros(n * page, dtype=torch.bool)
    keys = torch.full((n * page, d_rope), math.nan, dtype=torch.float64)
    pos = starts[:, None] + torch.arange(S)
    kk = cref.turn(cref.norm(k.double().cpu(), w.double().cpu(), 1e-6), pos[None], [d_rope // 2], 1e4, True) if d_rope else k.cpu()
    for b in range(B):
        for i in range(int(counts[b])):
            p = int(starts[b]) + i
            slot = int(table[b, p // page]) * page + p % page
            touched[slot] = True
            want_codes[slot] = torch.from_numpy(codes[b * S + i])
            want_scales[slot] = torch.from_numpy(scales[b * S + i])
            keys[slot] = kk[b, i]
    assert torch.equal(cache.scales.cpu().view(n * page, -1), want_scales)  # rows past the counts as they were
    assert torch.equal(cache.codes.cpu().view(n * page, -1), want_codes)
    got = cache.k_rope.double().cpu().view(n * page, d_rope)
    assert torch.equal(got.isnan(), keys.isnan())
    if d_rope:
        tol = 2.0 ** -8 if dtype == torch.bfloat16 else 80 * 2.0 ** -24
        assert float((got - keys)[touched].norm()) <= tol * float(keys[touched].norm())
    c, r = laga.cache4_read(cache, table, starts.int().to(dev()), S, counts=counts.int().to(dev()))
    inside = (torch.arange(S) < counts[:, None]).to(dev())
    want = torch.from_numpy(vals).view(B, S, d_c).to(dev())
    assert torch.equal(c.double()[inside], want[inside]) and not c[~inside].any() and not r[~inside].any()
    at = (torch.gather(table.cpu().long(), 1, pos.clamp(max=table.shape[1] * page - 1) // page) * page + pos % page).to(dev())
    assert torch.equal(r[inside], cache.k_rope.view(n * page, d_rope)[at[inside]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_scale_and_special_values(dtype):
    """One block for each scale of the grid and the values next to its border; infinities and NaN; saturation."""
    grid = cref.scale_values()[1:227]
    top = torch.tensor(6 * grid).to(dtype)
    up = torch.nextafter(top.float(), torch.tensor(math.inf)).to(dtype) if dtype == torch.float32 else \
        (top.view(torch.int16) + 1).view(dtype)
    x = torch.cat([top, up, torch.tensor([7e4, 3e38, math.inf, -math.inf, math.nan]).to(dtype)])
    rows = torch.zeros(x.numel(), 32, dtype=dtype)
    rows[:, 3], rows[:, 20] = x, -x
    rows[:, 5] = x / 24
    cache = pool(x.numel(), 1, 32, 0, dtype)
    table = torch.arange(x.numel(), dtype=torch.int32, device=dev())[None].contiguous()
    laga.cache4_append(cache, rows[None].to(dev()), torch.empty(1, x.numel(), 0, dtype=dtype, device=dev()), table, i32(0))
    codes, scales, vals = cref.encode(rows.double().numpy())
    assert np.array_equal(cache.scales.cpu().numpy()[:, 0], scales) and np.array_equal(cache.codes.cpu().numpy()[:, 0], codes)
    c, _ = laga.cache4_read(cache, table, i32(0), x.numel())
    c = c[0].double().cpu().numpy()
    assert np.array_equal(np.isnan(c), np.isnan(vals)) and np.array_equal(np.nan_to_num(c), np.nan_to_num(vals))
    assert abs(c[2 * 226 + 1]).max() == 61440 and np.isnan(c[-3:]).all()


def test_every_bf16_value_next_to_the_borders():
    """All bf16 values from an eighth of a scale to its largest multiple, both signs, for each form of a scale."""
    blocks = []
    for e in (1, 2, 3, 5, 7, 8, 9, 11, 15, *range(120, 128), 219, 225, 226):
        s = float(cref.scale_values()[e])
        lo, hi = (int(torch.tensor(v, dtype=torch.bfloat16).view(torch.int16)) for v in (s / 8, 6 * s))
        v = torch.arange(lo, hi + 1, dtype=torch.int16).view(torch.bfloat16)
        v = v[v.double() <= 6 * s]
        v = torch.cat([v, -v])
        v = torch.cat([v, v.new_zeros(-v.numel() % 15)]).view(-1, 15)
        blocks.append(torch.cat([v.new_full((v.shape[0], 1), 6 * s), v], 1))
    x = torch.cat(blocks)
    n = x.shape[0]
    cache = pool(n, 1, 16, 0, torch.bfloat16)
    table = torch.arange(n, dtype=torch.int32, device=dev())[None].contiguous()
    laga.cache4_append(cache, x[None].to(dev()), torch.empty(1, n, 0, dtype=torch.bfloat16, device=dev()), table, i32(0))
    codes, scales, _ = cref.encode(x.double().numpy())
    assert np.array_equal(cache.scales.cpu().numpy()[:, 0], scales) and np.array_equal(cache.codes.cpu().numpy()[:, 0], codes)


@pytest.mark.parametrize("d_c", [32, 20])
def test_bytes_past_the_largest_scale_are_not_finite(d_c):
    cache = laga.cache4(1, 256, d_c, 0, torch.float32, dev())
    cache.codes.fill_(0x21)
    cache.scales.copy_(torch.arange(256, device=dev(), dtype=torch.uint8)[None, :, None].expand_as(cache.scales))
    c, _ = laga.cache4_read(cache, torch.zeros(1, 1, dtype=torch.int32, device=dev()), i32(0), 256)
    assert torch.equal(c[0].isnan().all(1), torch.arange(256, device=dev()) > cref.TOP) and c[0, :cref.TOP + 1].isfinite().all()


def test_keys_turned_by_positions_of_several_axes():
    B, S, dr = 2, 13, 24
    cache = pool(8, 8, 32, dr, torch.float32)
    table = torch.arange(8, dtype=torch.int32, device=dev()).view(2, 4).contiguous()
    x, k = torch.randn(B, S, 32, device=dev()), torch.randn(B, S, dr, generator=gen(1), device=dev())
    pos = torch.randint(-9000, 9000, (3, B, S), generator=torch.Generator().manual_seed(2)).to(dev())
    for interleaved in (True, False):
        for p in (pos, pos.int()):
            laga.cache4_append(cache, x, k, table, i32(5, 0), pos=p, sections=[3, 4, 5], theta=5e5, interleaved=interleaved)
            _, r = laga.cache4_read(cache, table, i32(5, 0), S)
            want = cref.turn(k.double().cpu(), pos.cpu(), [3, 4, 5], 5e5, interleaved)
            assert float((r.double().cpu() - want).norm()) <= 80 * 2.0 ** -24 * float(want.norm())
    # as norm_rope leaves it, and stored as it comes
    w = torch.rand(dr, device=dev()) + 0.5
    _, kr = laga.norm_rope(None, k, pos, None, w, sections=[3, 4, 5])
    laga.cache4_append(cache, x, kr, table, i32(5, 0), theta=None)
    _, r = laga.cache4_read(cache, table, i32(5, 0), S)
    assert torch.equal(r, kr)


def test_positions_without_a_page():
    """They are left out, read as NaN, and reported; everything else is written."""
    cache = pool(6, 4, 32, 8, torch.float32)
    before = cache.codes.clone(), cache.scales.clone(), cache.k_rope.clone()
    table = torch.tensor([[0, 99], [-1, 2], [3, 4]], dtype=torch.int32, device=dev())
    x, k = torch.randn(3, 10, 32, device=dev()), torch.randn(3, 10, 8, device=dev())
    laga.check(dev())
    laga.cache4_append(cache, x, k, table, i32(0, 0, 6), theta=None)  # rows 2.. of the last run past its table
    with pytest.raises(laga.LagaError, match="page"):
        laga.check(dev())
    laga.check(dev())  # reported once
    c, r = laga.cache4_read(cache, table, i32(0, 0, 6), 10)
    with pytest.raises(laga.LagaError, match="page"):
        laga.check(dev())
    ok = torch.zeros(3, 10, dtype=torch.bool)
    ok[0, :4], ok[1, 4:8], ok[2, :2] = True, True, True
    assert c[~ok].isnan().all() and r[~ok].isnan().all() and c[ok].isfinite().all()
    assert torch.equal(r[ok], k[ok])
    for a, b in zip(before, (cache.codes, cache.scales, cache.k_rope)):  # pages 1, 3 and 5, half of 4
        for p in ((1,), (3,), (5,), (4, slice(0, 2))):
            same = torch.equal(a[p].view(torch.uint8), b[p].view(torch.uint8))
            assert same
    laga.cache4_append(cache, x, k, table, i32(-4, 0, 0), counts=i32(0, 0, 0))  # nothing to do, nothing wrong
    laga.check(dev())
    laga.cache4_append(cache, x, k, table, i32(-4, 0, 0), counts=i32(1, 0, 0), theta=None)
    with pytest.raises(laga.LagaError, match="page"):
        laga.check(dev())


# ---------------------------------------------------------------- attention
def queries(B, Sq, n_h, dims, dtype, seed=5, std=1.0):
    d_c, dn, dr, dv = dims
    g = gen(seed)
    q = (torch.randn(B, Sq, n_h, dn + dr, generator=g, device=dev()) * std).to(dtype)
    return q, *((torch.randn(d_c, n_h * d, generator=g, device=dev()) * d_c ** -0.5).to(dtype) for d in (dn, dv))


def slopes(n_h):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n_h) for h in range(n_h)], device=dev())


def compare(cache, table, lengths, q, W_UK, W_UV, tol=None, lse_tol=None, variant="auto", **kw):
    n = torch.as_tensor(lengths, dtype=torch.int32, device=dev())
    ws = laga.cache4_workspace(q, cache, W_UK, W_UV, table, variant=variant,
                               **{k: kw[k] for k in ("causal", "softmax_scale") if k in kw}).fill_(255)
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, workspace=ws, variant=variant, **kw)
    laga.check(dev())
    values = cref.decode(cache.codes, cache.scales, cache.d_c)
    kw["scale"] = kw.pop("softmax_scale", None)
    want = cref.attend(q, values, cache.k_rope, W_UK, W_UV, table, lengths, cache.page_size, **kw)
    tol = tol or TOL[q.dtype]
    got = {"out": out, "lse": lse}
    ref.close(got, want, tol, ("out",))
    empty = want["lse"] == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    err = (lse.double().cpu() - want["lse"])[~empty].abs()
    # a score's rounding in bf16 (2^-8 of the query's 512 latent values, of either sign: 2^-8 / sqrt(3) of the
    # score's own spread at most, five of them for the largest of a few thousand)
    bound = lse_tol or (5e-2 if q.dtype == torch.bfloat16 else 2e-5 + 8 * 2.0 ** -24 * want["lse"][~empty].abs())
    assert bool((err <= bound).all()), float(err.max())
    assert not out.cpu()[empty.transpose(1, 2)].any()
    return out, lse


MODS = {"plain": {}, "cap": dict(softcap=3.0), "bias": dict(slopes=True), "both": dict(softcap=8.0, slopes=True), "far": dict(softcap=3000.0),
        "far both": dict(softcap=900.0, slopes=True)}
CASES = {  # lengths, page, Sq, n_h
    "one": ([1], 1, 1, 1), "empty": ([0, 0], 4, 1, 2), "some": ([5, 0, 64, 65, 128], 16, 1, 3), "short": ([2, 7, 1], 16, 4, 2),
    "pages": ([300, 17, 129], 48, 3, 5), "rows": ([200, 131], 64, 9, 16), "wide": ([90, 411], 7, 2, 33), "long": ([3001], 128, 1, 16)}


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (64, 32, 16, 32)), (torch.float32, (37, 5, 6, 11)),
                                        (torch.bfloat16, (40, 24, 8, 16)), (torch.float32, (8, 3, 0, 1))])
def test_attention(dtype, dims, name, mod):
    lengths, page, Sq, n_h = CASES[name]
    cache, table = filled(lengths, page, dims, dtype)
    q, W_UK, W_UV = queries(len(lengths), Sq, n_h, dims, dtype)
    kw = dict(MODS[mod])
    if "slopes" in kw:
        kw["slopes"] = slopes(n_h)
    compare(cache, table, lengths, q, W_UK, W_UV, **kw)


@pytest.mark.parametrize("n_h", [1, 15, 16, 17, 31, 48, 64, 65, 100, 128, 130, 200, 256, 300])
def test_head_counts_bf16(n_h):
    lengths = [700, 1, 0, 129]
    cache, table = filled(lengths, 64, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(4, 1, n_h, DSV3, torch.bfloat16)
    compare(cache, table, lengths, q, W_UK, W_UV)


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (64, 32, 16, 32))])
@pytest.mark.parametrize("causal", [True, False])
def test_intervals_of_keys(dtype, dims, causal):
    """Any intervals, some empty, some past the ends; windows that skip whole tiles and pages."""
    lengths, Sq, n_h = [500, 40, 900], 6, 4
    cache, table = filled(lengths, 24, dims, dtype)
    q, W_UK, W_UV = queries(3, Sq, n_h, dims, dtype)
    g = torch.Generator().manual_seed(4)
    lo = torch.randint(-5, 890, (3, Sq), generator=g).int()
    hi = lo + torch.randint(-3, 400, (3, Sq), generator=g).int()
    hi[0, 2] = 0
    compare(cache, table, lengths, q, W_UK, W_UV, key_lo=lo.to(dev()), key_hi=hi.to(dev()), causal=causal)
    window = (torch.tensor(lengths)[:, None] - Sq + torch.arange(Sq) - 99).int().to(dev())
    compare(cache, table, lengths, q, W_UK, W_UV, key_lo=window, causal=causal)
    compare(cache, table, lengths, q, W_UK, W_UV, key_hi=hi.to(dev()), causal=causal, softmax_scale=0.3)


@pytest.mark.parametrize("n_h,lengths", [(16, [20000, 3, 9000]), (128, [15000, 700]), (40, [30000])])
def test_long_sequences_are_split_and_joined(n_h, lengths):
    cache, table = filled(lengths, 64, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(len(lengths), 1, n_h, DSV3, torch.bfloat16)
    out, lse = compare(cache, table, lengths, q, W_UK, W_UV)
    again = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(*lengths))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # the same bits


def test_many_short_sequences():
    g = torch.Generator().manual_seed(7)
    lengths = torch.randint(0, 300, (400,), generator=g).tolist()
    cache, table = filled(lengths, 32, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(400, 1, 16, DSV3, torch.bfloat16)
    compare(cache, table, lengths, q, W_UK, W_UV)


def test_a_whole_prompt_of_queries():
    cache, table = filled([333], 64, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(1, 333, 20, DSV3, torch.bfloat16)
    compare(cache, table, [333], q, W_UK, W_UV)
    cache, table = filled([90], 64, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(1, 130, 3, DSV3, torch.bfloat16)  # 40 rows before the first position
    compare(cache, table, [90], q, W_UK, W_UV)


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (64, 32, 16, 32))])
@pytest.mark.parametrize("what", ["latent", "key", "key_inf", "query", "query_inf"])
def test_values_that_are_not_finite(dtype, dims, what):
    """They reach the rows that see them, and no other: not their tile's, not their item's."""
    lengths, Sq, n_h = [200, 150], 4, 3
    cache, table = filled(lengths, 16, dims, dtype)
    q, W_UK, W_UV = queries(2, Sq, n_h, dims, dtype)
    n = i32(*lengths)
    clean = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n)
    bad = torch.zeros(2, Sq, n_h, dtype=torch.bool)
    p = 198  # seen by rows 2 and 3 of sequence 0
    page, at = int(table[0, p // 16]), p % 16
    if what == "latent":
        cache.scales[page, at, 1] = 255
        bad[0, 2:] = True
    elif what.startswith("key"):
        cache.k_rope[page, at, 3] = float("inf" if what == "key_inf" else "nan")
        bad[0, 2:] = True
    else:
        q[0, 1, 2, 7] = float("inf" if what == "query_inf" else "nan")
        bad[0, 1, 2] = True
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n)
    laga.check(dev())
    assert out.cpu()[bad].isnan().all() and lse.cpu().transpose(1, 2)[bad].isnan().all()
    assert torch.equal(out.cpu()[~bad], clean[0].cpu()[~bad])
    assert torch.equal(lse.cpu().transpose(1, 2)[~bad], clean[1].cpu().transpose(1, 2)[~bad])


@pytest.mark.parametrize("page", [5, 64])
@pytest.mark.parametrize("n_h", [6, 33])  # 24 and 132 rows a sequence: both forms of the tensor cores
def test_any_block_that_is_not_finite(n_h, page):
    """Each block of 16 and each key's place in a tile, one at a time: NaN in the rows that see it, bits as before elsewhere."""
    lengths, Sq = [203, 70], 4
    cache, table = filled(lengths, page, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(2, Sq, n_h, DSV3, torch.bfloat16)
    n = i32(*lengths)
    clean = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n)
    assert clean[0].isfinite().all()
    hi = torch.full((2, Sq), 2 ** 30, dtype=torch.int32, device=dev())
    hi[0, 2] = 40
    part = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, key_hi=hi)
    for k in range(64):
        p, block, byte = 3 * k + 13, (k * 11) % 32, (227, 254, 255)[k % 3]
        at = int(table[0, p // page]), p % page
        if k % 4 == 3:
            tensor, index, value = cache.k_rope, (*at, (5 * k) % 64), float(("nan", "inf", "-inf")[k % 3])
        else:
            tensor, index, value = cache.scales, (*at, block), byte
        was = tensor[index].clone()
        tensor[index] = value
        sees = torch.tensor([p <= lengths[0] - Sq + i for i in range(Sq)])
        for kw, want, rows in (({}, clean, sees), (dict(key_hi=hi), part, sees & torch.tensor([True, True, p < 40, True]))):
            out, lse = (t.cpu() for t in laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, **kw))
            assert out[0, rows].isnan().all() and lse[0][:, rows].isnan().all(), (p, k)
            assert torch.equal(out[0, ~rows], want[0].cpu()[0, ~rows]) and torch.equal(out[1], want[0].cpu()[1]), (p, k)
        tensor[index] = was
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    laga.check(dev())


@pytest.mark.parametrize("n_h", [6, 33])
def test_pages_missing_inside(n_h):
    """Entries that are no page: NaN for the rows that see their keys, whatever else the tile holds."""
    lengths, Sq, page = [203, 70], 4, 7
    cache, table = filled(lengths, page, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(2, Sq, n_h, DSV3, torch.bfloat16)
    n = i32(*lengths)
    hi = torch.full((2, Sq), 2 ** 30, dtype=torch.int32, device=dev())
    hi[0, 1] = 60
    clean = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, key_hi=hi)
    laga.check(dev())
    for entry, value in ((9, -1), (14, 10 ** 6), (28, -2 ** 31), (20, 2 ** 31 - 1)):
        broken = table.clone()
        broken[0, entry] = value
        out, lse = (t.cpu() for t in laga.cache4_fwd(q, cache, W_UK, W_UV, broken, n, key_hi=hi))
        with pytest.raises(laga.LagaError, match="page"):
            laga.check(dev())
        rows = torch.tensor([True, entry * page < 60, True, True])
        assert out[0, rows].isnan().all() and lse[0][:, rows].isnan().all()
        assert torch.equal(out[0, ~rows], clean[0].cpu()[0, ~rows]) and torch.equal(out[1], clean[0].cpu()[1])


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (64, 32, 16, 32))])
def test_tables_that_do_not_hold_the_sequence(dtype, dims):
    lengths = [100, 100, 100]
    cache, table = filled(lengths, 16, dims, dtype)
    q, W_UK, W_UV = queries(3, 2, 4, dims, dtype)
    clean = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(*lengths))
    broken = table.clone()
    broken[0, 2] = 10 ** 6
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, broken, i32(100, 100, 113))
    with pytest.raises(laga.LagaError, match="page"):
        laga.check(dev())
    assert out[0].isnan().all() and lse[0].isnan().all() and out[2].isnan().all() and lse[2].isnan().all()
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(2 ** 31 - 1, 100, -7))
    with pytest.raises(laga.LagaError, match="page"):
        laga.check(dev())
    assert out[0].isnan().all() and torch.equal(out[1], clean[0][1])
    assert not out[2].any() and (lse[2] == -math.inf).all()


def test_large_and_small_scores_bf16():
    """Scores of hundreds (one key takes all), of 1e-6, and latents at both ends of the format."""
    for std_q, std_c in ((30.0, 1.0), (1e-6, 1.0), (1e-3, 2000.0), (300.0, 2.0 ** -12)):
        cache, table = filled([700, 90], 64, DSV3, torch.bfloat16, std=std_c)
        q, W_UK, W_UV = queries(2, 2, 20, DSV3, torch.bfloat16, std=std_q)
        # a score's error, 2^-8 / sqrt(3) of its size in the root mean square, acts on the weight in proportion
        size = max(1.0, std_q * std_c)
        compare(cache, table, [700, 90], q, W_UK, W_UV, tol=TOL[torch.bfloat16] * max(1.0, size / 2), lse_tol=5e-2 * size)


def test_captured_with_new_lengths_and_tables():
    """One graph serves growing sequences: lengths and pages are read at the replay."""
    cache, table = filled([900, 300, 64], 64, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(3, 1, 16, DSV3, torch.bfloat16)
    n = i32(100, 0, 64)
    t = table.clone()
    ws = laga.cache4_workspace(q, cache, W_UK, W_UV, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        laga.cache4_fwd(q, cache, W_UK, W_UV, t, n, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, t, n, workspace=ws)
    for lengths, order in (([100, 0, 64], [0, 1, 2]), ([900, 300, 1], [0, 1, 2]), ([290, 850, 0], [1, 0, 2])):
        n.copy_(i32(*lengths))
        t.copy_(table[order])
        q.mul_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = laga.cache4_fwd(q, cache, W_UK, W_UV, t, n)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        compare(cache, t, lengths, q, W_UK, W_UV)


def test_two_calls_at_once():
    cache, table = filled([5000, 3000], 64, DSV3, torch.bfloat16)
    sets = [queries(2, 1, n_h, DSV3, torch.bfloat16, seed=n_h) for n_h in (16, 128)]
    n = i32(5000, 3000)
    want = [laga.cache4_fwd(s[0], cache, s[1], s[2], table, n) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k].append(laga.cache4_fwd(s[0], cache, s[1], s[2], table, n))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, want[k][0]) and torch.equal(l, want[k][1]) for o, l in got[k])


@pytest.mark.parametrize("dtype,dims", [(torch.bfloat16, DSV3), (torch.float32, (64, 32, 16, 32))])
def test_prompt_then_tokens(dtype, dims):
    """As a server runs them: a prompt appended (its attention rebuilt from the cache's values by masked_fwd), then
    tokens one at a time through norm_rope, append and attention, each against the definition in 64 bits."""
    d_c, dn, dr, dv = dims
    B, n_h, page, steps = 2, 5, 16, 4
    prompt = [37, 20]
    g = gen(21)

    def normal(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g, device=dev()) * std + mean).to(dtype)
    wq, wk = normal(dn + dr, std=0.2, mean=1.0), normal(dr, std=0.2, mean=1.0)
    W_UK, W_UV = normal(d_c, n_h * dn, std=d_c ** -0.5), normal(d_c, n_h * dv, std=d_c ** -0.5)
    table, pages = tables([n + steps for n in prompt], page)
    cache = pool(pages, page, d_c, dr, dtype)
    S = max(prompt)
    q, c, k = normal(B, S, n_h, dn + dr, std=3.0), normal(B, S, d_c), normal(B, S, dr, std=2.0)
    counts, zero = i32(*prompt), i32(0, 0)
    pos = torch.arange(S, device=dev(), dtype=torch.int32).expand(1, B, S).contiguous()
    qr, _ = laga.norm_rope(q, None, pos, wq, sections=[dr // 2])
    laga.cache4_append(cache, c, k, table, zero, counts=counts, k_weight=wk)
    c4, kr = laga.cache4_read(cache, table, zero, S, counts=counts)
    lo, hi = laga.key_bounds(torch.stack([zero, counts], 1).contiguous(), S)
    out, _ = laga.masked_fwd(qr, c4, kr, W_UK, W_UV, key_lo=lo, key_hi=hi)
    values = cref.decode(cache.codes, cache.scales, d_c)
    yq, _ = cref.norm_rope(q.double().cpu(), None, pos.cpu(), wq.double().cpu(), None, 1e-6, [dr // 2], 1e4, True)
    # norm_rope's rounding of q and the masked forward's four: five of 2.3e-3, doubled for scores above 1
    tol = 2 * 5 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 if dtype == torch.bfloat16 else 2 * TOL[dtype]
    for b in range(B):
        want = cref.attend(yq[b:b + 1, :prompt[b]], values, cache.k_rope, W_UK, W_UV, table[b:b + 1], [prompt[b]], page)
        ref.close({"out": out[b:b + 1, :prompt[b]]}, want, tol, ("out",))
        direct, _ = laga.cache4_fwd(qr[b:b + 1, :prompt[b]].contiguous(), cache, W_UK, W_UV, table[b:b + 1], counts[b:b + 1])
        ref.close({"out": direct}, want, tol, ("out",))
    lengths = counts.clone()
    for _ in range(steps):
        q, c, k = normal(B, 1, n_h, dn + dr, std=3.0), normal(B, 1, d_c), normal(B, 1, dr, std=2.0)
        at = lengths[None, :, None].clone()
        qr, _ = laga.norm_rope(q, None, at, wq, sections=[dr // 2])
        laga.cache4_append(cache, c, k, table, lengths, k_weight=wk)
        lengths += 1
        out, lse = laga.cache4_fwd(qr, cache, W_UK, W_UV, table, lengths)
        yq, _ = cref.norm_rope(q.double().cpu(), None, at.cpu(), wq.double().cpu(), None, 1e-6, [dr // 2], 1e4, True)
        want = cref.attend(yq, cref.decode(cache.codes, cache.scales, d_c), cache.k_rope, W_UK, W_UV, table,
                           lengths.tolist(), page)
        ref.close({"out": out}, want, tol, ("out",))
    laga.check(dev())


def test_nothing_and_argument_checks():
    cache, table = filled([40, 20], 16, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(2, 1, 4, DSV3, torch.bfloat16)
    n = i32(40, 20)
    out, lse = laga.cache4_fwd(q[:, :0].contiguous(), cache, W_UK, W_UV, table, n)
    assert out.shape == (2, 0, 4, 128) and lse.shape == (2, 4, 0)
    c, k = laga.cache4_read(cache, table, n, 0)
    assert c.shape == (2, 0, 512) and k.shape == (2, 0, 64)
    laga.cache4_append(cache, c, k, table, n)
    with pytest.raises(ValueError, match="lengths"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table, n[:1])
    with pytest.raises(TypeError, match="lengths"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table, n.long())
    with pytest.raises(ValueError, match="table"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table[:1], n)
    with pytest.raises(ValueError, match="row for each latent"):
        laga.cache4_fwd(q, cache, W_UK[:64], W_UV, table, n)
    with pytest.raises(ValueError, match="d_rope"):
        laga.cache4_fwd(q[..., :160].contiguous(), cache, W_UK, W_UV, table, n)
    with pytest.raises(TypeError):
        laga.cache4_fwd(q.float(), cache, W_UK, W_UV, table, n)
    with pytest.raises(laga.LagaError, match="softcap"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, softcap=-1.0)
    with pytest.raises(laga.LagaError, match="variants"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, variant="fused_recon")
    with pytest.raises(ValueError, match="workspace"):
        laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, workspace=torch.empty(8, device=dev()))
    with pytest.raises(ValueError, match="pos"):
        laga.cache4_append(cache, c, k, table, n, pos=torch.zeros(1, 2, 0, dtype=torch.int32, device=dev()), theta=None)
    with pytest.raises(ValueError, match="cache.scales"):
        laga.cache4_read(laga.Cache4(cache.codes, cache.scales[..., :31].contiguous(), cache.k_rope, 512), table, n, 1)


def test_bf16_on_the_cuda_cores():
    cache, table = filled([300, 77], 16, DSV3, torch.bfloat16)
    q, W_UK, W_UV = queries(2, 3, 10, DSV3, torch.bfloat16)
    # inputs and result rounded alone
    compare(cache, table, [300, 77], q, W_UK, W_UV, tol=2.0 ** -8, lse_tol=1e-4, variant="simt")
