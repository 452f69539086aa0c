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


@pytest.mark.parametrize("dtype,dims", KINDS)
@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("seen_by_padding", [False, True])
def test_keys_outside_the_documents(dtype, dims, value, cap, seen_by_padding):
    """The padding's latents, RoPE keys, q and dout are huge; seen_by_padding: and a document of its own, whose
    results (and with them the weights' gradients) are anything."""
    x, dout, kw = packed(dtype, dims, seen_by_padding)
    kw["softcap"] = cap
    want = step(x, dout, **kw)
    y, dy = {k: v.clone() for k, v in x.items()}, dout.clone()
    for b, end in ENDS:
        y["c_kv"][b, end:] = value
        y["k_rope"][b, end:, ::3] = -value
        y["q"][b, end:] = value
        dy[b, end:] = value
    got = step(y, dy, **kw)
    same_rows(got, want, ("dW_UK", "dW_UV") if seen_by_padding else ())
    if not seen_by_padding:
        for b, end in ENDS:
            assert not got["dc_kv"][b, end:].any() and not got["dk_rope"][b, end:].any()
    laga.check(dev())


@pytest.mark.parametrize("dtype,dims", KINDS[:2])
def test_a_row_that_sees_a_key_out_of_range(dtype, dims):
    """A latent value above 2^112 counts as not finite: the rows that see its key get NaN, no others; at 2^112
    it is a value like any other."""
    x, dout, kw = packed(dtype, dims)
    want = step(x, dout, **kw)
    y = {k: v.clone() for k, v in x.items()}
    y["c_kv"][0, 150, 5] = 1.5 * 2.0 ** 112
    got = step(y, dout, **kw)
    hit = torch.zeros(B, S, dtype=torch.bool, device=dev())
    hit[0, 150:230] = True
    assert got["out"][hit].isnan().all() and torch.equal(got["out"][~hit], want["out"][~hit])
    assert got["dq"][hit].isnan().all() and torch.equal(got["dq"][~hit], want["dq"][~hit])
    y["c_kv"][0, 150, 5] = -2.0 ** 112
    y["W_UK"][5] = 0.0  # its scores stay small; its V does not
    y["W_UV"][5] = 2.0 ** -112
    out, lse = laga.masked_fwd(*y.values(), **kw)
    assert bool(out[hit].isfinite().all()) and bool(lse[0, :, 150:230].isfinite().all())
    laga.check(dev())
