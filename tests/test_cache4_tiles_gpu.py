"""The cache attention over many key tiles a part: the running maximum moved within a piece, masks, biases and places that
are not finite past a piece's first tile, and the precision that the tensor-core forms keep between their products.
Against the definition in 64 bits, in every form.

Tolerances, in the 2-norm relative to the result. A rounding's root mean square is its half step over sqrt(3).
bf16 forms on the tensor cores: the result 2^-8, the weights 2^-11 (fp16), and the query in the latent space 2^-11, which
moves a score by `e` = 2^-11 / sqrt(3) of the latent part's own spread, 0.82 (128 values of W_UK of size 512^-1/2 a
column, 512 columns, over sqrt(192)) times the size of the queries; weights follow the difference of two scores, at most
2 e. A quarter is added, for sums of a few thousand values of which not all are alike. The log of the sum is not rounded:
six e, and 3e-4 for 36 steps of the products' sums of up to 60 in fp32.
CUDA cores: sums of D values of up to S, 2^-24 sqrt(D) S for each score, and as many again for all that follows; the
plain tolerance of test_cache4_gpu.py (100 * 2^-24, doubled) beside it; in bf16 the result's 2^-8."""
import functools
import math

import pytest
import torch

from mla_attention_sequence_gb300 import laga
from test_cache4_gpu import DSV3, built, dev, gen, i32, pool, queries, slopes, tables  # noqa: F401
from test_cache4_rows_gpu import latent_attention, lost, stored

pytestmark = pytest.mark.gpu
SQ = 2
FORMS = {  # type, widths, heads, lengths, keys of a tile, rows of a tile, CTAs that share the tiles for each SM
    "fp32": (torch.float32, (64, 32, 16, 32), 40, [6400, 300], 32, 8, 2),
    "bf16 on the CUDA cores": (torch.bfloat16, (40, 24, 8, 16), 40, [6400, 300], 32, 8, 2),
    "mma.sync": (torch.bfloat16, DSV3, 16, [30000, 21000], 32, 16, 2), "tcgen05": (torch.bfloat16, DSV3, 40, [26000, 100], 64, 128, 0.5)}
PAGE = 24
MODS = {"plain": {}, "cap": dict(softcap=3.0), "bias": dict(slopes=True), "both": dict(softcap=8.0, slopes=True),
        "far": dict(softcap=3000.0), "far both": dict(softcap=900.0, slopes=True), "interval": dict(interval=True),
        "interval, both": dict(interval=True, softcap=8.0, slopes=True)}


@functools.lru_cache(maxsize=None)
def data(form, how):
    """Tokens whose RoPE keys grow or shrink along the sequence (scores up to some 50, from 0), or queries of size 8."""
    dtype, (d_c, dn, dr, dv), n_h, lengths, keys, rows, ctas = FORMS[form]
    # five tiles a part at least, so that most pieces have several
    parts = int(torch.cuda.get_device_properties(0).multi_processor_count * ctas)
    assert sum(n // keys * -(-SQ * n_h // rows) for n in lengths) >= 5 * parts
    table, pages = tables(lengths, PAGE)
    cache = pool(pages, PAGE, d_c, dr, dtype)
    most = max(lengths)
    x = torch.randn(2, most, d_c, generator=gen(1), device=dev()).to(dtype)
    j = torch.arange(most, device=dev())[None, :, None] / torch.tensor(lengths, device=dev())[:, None, None]
    size = {"up": 20 * j, "down": 20 * (1 - j), "size 8": torch.ones_like(j)}[how]
    k = (torch.randn(2, most, dr, generator=gen(2), device=dev()) * size).to(dtype)
    laga.cache4_append(cache, x, k, table, i32(0, 0), counts=i32(*lengths), theta=None)
    q, W_UK, W_UV = queries(2, SQ, n_h, (d_c, dn, dr, dv), dtype, std=8.0 if how == "size 8" else 1.0)
    return cache, table, q, W_UK, W_UV, [stored(cache, table, b, n) for b, n in enumerate(lengths)]


def tolerances(form, how):
    dtype, (d_c, dn, dr, dv), *_ = FORMS[form]
    if form in ("mma.sync", "tcgen05"):
        e = 2.0 ** -11 / 3 ** 0.5 * 0.82 * (8 if how == "size 8" else 1)
        return 1.25 * math.sqrt((2.0 ** -16 + 2.0 ** -22) / 3 + (2 * e) ** 2), 6 * e + 3e-4
    S = 60
    each = 2.0 ** -24 * math.sqrt(d_c + dr) * S
    return 200 * 2.0 ** -24 + 2 * each + (2.0 ** -8 if dtype == torch.bfloat16 else 0), 2e-5 + 3 * each


@pytest.mark.parametrize("how", ["up", "down", "size 8"])
@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("form", FORMS)
def test_pieces_of_several_tiles(form, mod, how):
    n_h, lengths = FORMS[form][2:4]
    cache, table, q, W_UK, W_UV, held = data(form, how)
    kw = dict(MODS[mod])
    if kw.pop("slopes", False):
        kw["slopes"] = slopes(n_h)
    lo = torch.zeros(2, SQ, dtype=torch.int32)
    hi = torch.tensor([[n - SQ + i + 1 for i in range(SQ)] for n in lengths], dtype=torch.int32)
    call = dict(kw)
    if call.pop("interval", False):
        lo = torch.tensor([[n // 3 + 7, n // 2 + 1] for n in lengths], dtype=torch.int32)
        hi = torch.tensor([[n - 5, n - n // 5] for n in lengths], dtype=torch.int32)
        call.update(key_lo=lo.to(dev()), key_hi=hi.to(dev()))
    kw.pop("interval", None)
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(*lengths), **call)
    again = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(*lengths), **call)
    laga.check(dev())
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # the same bits
    tol, lse_tol = tolerances(form, how)
    for b, n in enumerate(lengths):
        want = latent_attention(q[b], *held[b], W_UK, W_UV, lo[b], hi[b], pos=n - SQ + torch.arange(SQ), **kw)
        err = float((out[b].double() - want[0]).norm() / want[0].norm())
        assert err <= tol, (b, err, tol)
        err = float((lse[b].double() - want[1]).abs().max())
        assert err <= lse_tol, (b, err, lse_tol)


@pytest.mark.parametrize("form", FORMS)
def test_places_that_are_not_finite_in_any_tile(form):
    """Blocks, RoPE keys and pages that are not there, one at a time, at both ends of tiles and pieces: NaN in the rows that
    see them, bits as before elsewhere."""
    dtype, dims, n_h, lengths, *_ = FORMS[form]
    cache, table, q, W_UK, W_UV, _ = data(form, "up")
    n, L = i32(*lengths), lengths[0]
    hi = i32(L // 2, 2 ** 30, 2 ** 30, 2 ** 30).view(2, SQ)
    clean = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, key_hi=hi)
    assert clean[0].isfinite().all()
    at = [0, 31, 32, 63, 64, 191, 192, 1000, L // 3, L // 2 - 1, L // 2, L // 2 + 77, L - 65, L - 2, L - 1]
    for k, p in enumerate(at):
        broken, page = table, int(table[0, p // PAGE])
        index = (page, p % PAGE)
        was = cache.scales[index].clone(), cache.k_rope[index].clone()
        if k % 3 == 0:
            cache.scales[index][(5 * k) % was[0].numel()] = 227 + k
        elif k % 3 == 1:
            cache.k_rope[index][(7 * k) % was[1].numel()] = math.nan if k % 2 else -math.inf
        else:
            broken = table.clone()
            broken[0, p // PAGE] = -1 if k % 2 else 2 ** 30
        out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, broken, n, key_hi=hi)
        first = p if k % 3 < 2 else p // PAGE * PAGE  # the place, or the first of the page
        rows = [first < L // 2, first < L]
        if k % 3 == 2:
            with pytest.raises(laga.LagaError, match="page"):
                laga.check(dev())
        for i in range(SQ):
            if rows[i]:
                assert lost(out[0], lse[0], [i]), (p, i)
            else:
                assert torch.equal(out[0, i], clean[0][0, i]) and torch.equal(lse[0, :, i], clean[1][0, :, i]), (p, i)
        assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1]), p
        cache.scales[index], cache.k_rope[index] = was
    out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, key_hi=hi)
    laga.check(dev())
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("n_h", [8, 80])  # mma.sync and tcgen05
def test_the_context_keeps_sixteen_bits(n_h):
    """Two latent columns that are nearly always alike, with opposite weights: the result is a difference of some 0.012 of
    two contexts of 4, of which one rounding to bf16 (steps of 2^-5 there) would leave nothing. Two parts leave steps of
    2^-14 at most, half of one for each column, 2^-15 sqrt(2) / 0.012 = 0.4% of the result; its own rounding is 2^-8; 190 steps of the
    products' sums lose at most 2^-23 of 4 each, 0.8%."""
    L = 3000
    table, pages = tables([L], 64)
    cache = pool(pages, 64, 512, 64, torch.bfloat16)
    x = torch.randn(1, L, 512, generator=gen(1), device=dev())
    x[..., :32] = 0
    x[..., 1] = x[..., 17] = 6.0  # the scale of both blocks: 1
    for c, seed in ((0, 2), (16, 3)):
        x[..., c] = torch.where(torch.rand(1, L, generator=gen(seed), device=dev()) < 0.02, 6.0, 4.0)
    k = torch.randn(1, L, 64, generator=gen(4), device=dev())
    laga.cache4_append(cache, x.bfloat16(), k.bfloat16(), table, i32(0), theta=None)
    q, W_UK, W_UV = queries(1, 1, n_h, DSV3, torch.bfloat16)
    W_UV.zero_()
    W_UV[0] = torch.randn(W_UV.shape[1], generator=gen(5), device=dev()).bfloat16()
    W_UV[16] = -W_UV[0]
    values, keys = stored(cache, table, 0, L)
    assert set(values[:, 0].tolist()) == {4.0, 6.0}
    out, _ = laga.cache4_fwd(q, cache, W_UK, W_UV, table, i32(L))
    laga.check(dev())
    want, _ = latent_attention(q[0], values, keys, W_UK, W_UV, [0], [L])
    err = float((out[0].double() - want).norm() / want.norm())
    assert err <= 2.0 ** -8 + 2.0 ** -15 * 2 ** 0.5 / 0.012 + 190 * 2.0 ** -23 * 4 / 0.012, err
