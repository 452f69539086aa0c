"""Rows of the cache attention that stand beside others in a tile, in every form."""
import math

import pytest
import torch

from mla_attention_sequence_gb300 import laga
from test_cache4_gpu import DSV3, built, dev, filled, i32, queries  # noqa: F401

pytestmark = pytest.mark.gpu
# type, widths, heads, variant: CUDA cores twice, mma.sync (up to 32 rows a sequence), tcgen05
FORMS = {"fp32": (torch.float32, (64, 32, 16, 32), 3, "auto"), "bf16 on the CUDA cores": (torch.bfloat16, DSV3, 3, "simt"),
         "mma.sync": (torch.bfloat16, DSV3, 3, "auto"), "tcgen05": (torch.bfloat16, DSV3, 40, "auto")}


def empty(out, lse, rows):
    return not out[rows].any() and bool((lse[:, rows] == -math.inf).all())


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
