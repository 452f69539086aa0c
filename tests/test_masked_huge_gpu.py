"""Masked attention with finite but huge values in masked places, as uninitialised padding or a mask by the
type's lowest value leaves them: what does not see them, and is not seen by them, keeps its results to the bit."""
import pytest
import torch

from mla_attention_sequence_gb300 import laga

from test_masked_gpu import DSV3, built, dev, inputs, step  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [(torch.bfloat16, DSV3), (torch.float32, (32, 16, 8, 24)), (torch.float32, (48, 100, 28, 130))]
HUGE = [3e38, -3.3e38, 1e33]
ENDS = ((0, 230), (1, 251))  # where the documents of each batch element end; the rest is padding
B, S, H = 2, 260, 2


def packed(dtype, dims, docs_of_padding=False):
    starts = [[0, 100, 230], [0, 31, 251]]
    if docs_of_padding:
        starts = [s + [S] for s in starts]
    lo, hi = laga.key_bounds(torch.tensor(starts, dtype=torch.int32, device=dev()), S)
    x, dout = inputs(B, S, S, H, dims, dtype, 71)
    return x, dout, dict(key_lo=lo, key_hi=hi)


def same_rows(got, want, skip=()):
    """Rows and keys of the documents, to the bit."""
    for k in want:
        if k in skip:
            continue
        if k.startswith("dW"):
            assert torch.equal(got[k], want[k]), k
            continue
        for b, end in ENDS:
            a, w = (t[k][b, :, :end] if k == "lse" else t[k][b, :end] for t in (got, want))
            assert torch.equal(a, w), k


@pytest.mark.parametrize("dtype,dims", KINDS)
@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_dout_of_rows_that_see_nothing(dtype, dims, value, cap):
    x, dout, kw = packed(dtype, dims)
    kw["softcap"] = cap
    want = step(x, dout, **kw)
    dy = dout.clone()
    for b, end in ENDS:
        dy[b, end:] = value
    got = step(x, dy, **kw)
    same_rows(got, want)
    for b, end in ENDS:
        assert not got["out"][b, end:].any() and not got["dq"][b, end:].any()
    laga.check(dev())


@pytest.mark.parametrize("dtype,dims", KINDS)
@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("cap", [0.0, 9.0, 600.0])
def test_q_of_rows_that_see_nothing(dtype, dims, value, cap):
    x, dout, kw = packed(dtype, dims)
    kw["softcap"] = cap
    want = step(x, dout, **kw)
    y = {k: v.clone() for k, v in x.items()}
    for b, end in ENDS:
        y["q"][b, end:] = value
        y["q"][b, end:, :, ::2] = -value  # products of both signs: their sums may be NaN
    got = step(y, dout, **kw)
    same_rows(got, want)
    for b, end in ENDS:
        assert not got["out"][b, end:].any() and not got["dq"][b, end:].any()
    laga.check(dev())
