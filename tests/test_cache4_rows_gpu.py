"""Rows of the cache attention that stand beside others in a tile: rows that see nothing and hold anything, rows that see
past the table beside rows that do not. Against the definition in 64 bits (in the latent space), in every form."""
import math

import pytest
import torch

import cache4_reference as cref
from mla_attention_sequence_gb300 import laga
from test_cache4_gpu import DSV3, TOL, built, dev, filled, i32, queries  # noqa: F401

pytestmark = pytest.mark.gpu
# type, widths, heads, variant: CUDA cores twice, mma.sync (up to 32 rows a sequence), tcgen05
FORMS = {"fp32": (torch.float32, (64, 32, 16, 32), 3, "auto"), "bf16 on the CUDA cores": (torch.bfloat16, DSV3, 3, "simt"),
         "mma.sync": (torch.bfloat16, DSV3, 3, "auto"), "tcgen05": (torch.bfloat16, DSV3, 40, "auto")}


def latent_attention(q, values, keys, W_UK, W_UV, lo, hi, softcap=0.0, slopes=None, pos=None, scale=None):
    """out [Sq, n_h, d_v], lse [n_h, Sq] of one sequence's queries over values [n, d_c], keys [n, d_rope] in 64 bits: row i
    sees lo[i] <= j < hi[i]. In the latent space, on the GPU."""
    q, values, keys, W_UK, W_UV = (t.to(dev()).double() for t in (q, values, keys, W_UK, W_UV))
    Sq, n_h, d_qk = q.shape
    d_c, d_rope = values.shape[1], keys.shape[1]
    d_nope, j = d_qk - d_rope, torch.arange(values.shape[0], device=dev())
    lat = torch.einsum("shd,chd->shc", q[..., :d_nope], W_UK.view(d_c, n_h, d_nope))
    s = (lat @ values.T + q[..., d_nope:] @ keys.T) * (scale or d_qk ** -0.5)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    if slopes is not None:
        s = s - slopes.double()[None, :, None] * (pos.to(dev())[:, None] - j).abs()[:, None, :]
    lo, hi = (torch.as_tensor(t, device=dev()).long()[:, None, None] for t in (lo, hi))
    s = torch.where((j >= lo) & (j < hi), s, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return torch.einsum("shc,chv->shv", w @ values, W_UV.view(d_c, n_h, -1)), lse.T


def stored(cache, table, b, n):
    """The n values and keys of sequence b that the cache's bytes stand for."""
    ids = table[b, :-(-n // cache.page_size)].long().cpu()
    values = cref.decode(cache.codes.cpu()[ids], cache.scales.cpu()[ids], cache.d_c)
    return values.flatten(0, 1)[:n].to(dev()), cache.k_rope.double()[ids.to(dev())].flatten(0, 1)[:n]


def near(out, lse, want, rows, dtype):
    """Those rows (of one sequence) against `want`, in the 2-norm of the whole; none of them -inf."""
    a, b = out.double()[rows], want[0][rows]
    assert float((a - b).norm()) <= TOL[dtype] * float(b.norm())
    assert bool(((lse.double() - want[1])[:, rows].abs() <= (5e-2 if dtype == torch.bfloat16 else 1e-4)).all())


def empty(out, lse, rows):
    return not out[rows].any() and bool((lse[:, rows] == -math.inf).all())


def lost(out, lse, rows):
    return bool(out[rows].isnan().all()) and bool(lse[:, rows].isnan().all())


@pytest.mark.parametrize("form", FORMS)
def test_rows_that_see_nothing_may_hold_anything(form):
    """Zero and -inf, whatever their queries and their tile's other rows are; the others keep their bits. Sequences that
    one part holds whole, and one that many share."""
    dtype, dims, n_h, variant = FORMS[form]
    lengths, Sq = [2, 300, 20000], 5
    cache, table = filled(lengths, 16, dims, dtype)
    q, W_UK, W_UV = queries(3, Sq, n_h, dims, dtype)
    hi = torch.full((3, Sq), 2 ** 30, dtype=torch.int32, device=dev())
    hi[1, 3] = hi[2, 1] = 0
    none = torch.zeros(3, Sq, dtype=torch.bool)
    none[0, :3] = none[1, 3] = none[2, 1] = True  # before the first position, and an interval of no keys
    n = i32(*lengths)

    def call(q):
        out, lse = laga.cache4_fwd(q, cache, W_UK, W_UV, table, n, key_hi=hi, variant=variant)
        laga.check(dev())
        return out.cpu(), lse.cpu()
    clean = call(q)
    assert clean[0].isfinite().all()
    for value in (math.nan, math.inf, -math.inf):
        for col in (0, dims[1] + dims[2] - 1, slice(None)):  # the part without positions, the RoPE part, all
            bad = q.clone()
            for b, i in none.nonzero().tolist():
                bad[b, i, :, col] = value
            out, lse = call(bad)
            for b in range(3):
                assert empty(out[b], lse[b], none[b]), (value, col, b)
            assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1]), (value, col)


@pytest.mark.parametrize("form", FORMS)
def test_rows_beside_rows_that_see_past_the_table(form):
    """NaN for the rows that see a position that the table has no room for, and for no other row of their tile."""
    dtype, dims, n_h, variant = FORMS[form]
    full, Sq = [112, 20000], 3  # to the last place of their last page
    cache, table = filled(full, 16, dims, dtype)
    tables = [table[:1, :7].contiguous(), table[1:].contiguous()]
    q, W_UK, W_UV = queries(2, Sq, n_h, dims, dtype)
    far = 2 ** 31 - 1
    for b in range(2):
        m = full[b]
        values, keys = stored(cache, table, b, m)
        # (length, key_lo, key_hi) or None; rows that are lost; rows that see nothing
        for length, lo, hi, gone, none in ((m + 1, None, None, [2], []), (m + 2, None, None, [1, 2], []),
                                           (far, [0, 0, 0], [m, 0, far], [2], [1]), (far, [0, m - 1, 5], [m - 1, m, m + 1], [2], []),
                                           (m + 900, [m + 1, m + 500, 0], [m + 2, far, 0], [0, 1], [2]),
                                           (m + 900, [0, m + 500, 5], [50, m + 700, m], [1], []),
                                           (m + 900, [m] * 3, [m + 900] * 3, [0, 1, 2], []),
                                           # keys past the room in the last tile that has others in it
                                           (m + 900, [0, m + 3, 5], [50, m + 9, m], [1], []),
                                           (m + 900, [m - 5, m + 1, 0], [m, m + 2, 0], [1], [2]),
                                           (m + 900, [m + 2, m, m + 1], [m + 40, m + 1, far], [0, 1, 2], [])):
            kw = {} if lo is None else dict(key_lo=i32(*lo)[None], key_hi=i32(*hi)[None])
            out, lse = laga.cache4_fwd(q[b:b + 1], cache, W_UK, W_UV, tables[b], i32(length), variant=variant, **kw)
            with pytest.raises(laga.LagaError, match="page"):
                laga.check(dev())
            at = [min(h, length - Sq + i + 1) for i, h in enumerate(hi or [far] * 3)]
            want = latent_attention(q[b], values, keys, W_UK, W_UV, lo or [0] * 3, at)
            case = (b, length, lo, hi)
            assert not gone or lost(out[0], lse[0], gone), case
            assert not none or empty(out[0], lse[0], none), case
            rows = [i for i in range(Sq) if i not in gone + none]
            if rows:
                near(out[0], lse[0], want, rows, dtype)
