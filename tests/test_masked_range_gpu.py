"""Masked attention where scores and values lie far from 1."""
import pytest
import torch

import masked_reference as ref
from mla_attention_sequence_gb300 import laga

from test_masked_gpu import DSV3, TOL, built, check, dev, inputs, random_bounds, slopes  # noqa: F401

pytestmark = pytest.mark.gpu


def forward(x, lo, hi, **kw):
    B, Sq = x["q"].shape[:2]
    S = x["c_kv"].shape[1]
    seen = ref.visible(Sq, S, lo, hi, causal=False, B=B)
    want = ref.attention(x, seen, kw.get("softcap", 0.0), kw.get("slopes"), pos=torch.arange(Sq))
    out, lse = laga.masked_fwd(*x.values(), key_lo=lo, key_hi=hi, causal=False, **kw)
    laga.check(dev())
    ref.close({"out": out}, want, TOL[torch.bfloat16], ("out",))
    empty = want["lse"] == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    assert float((lse.double() - want["lse"])[~empty].abs().max()) <= 5e-2


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("S", [300, 8300])
@pytest.mark.parametrize("level,size", [(62.0, 36), (62.0, 0), (-62.0, -40), (-62.0, 36), (20.0, 80), (-20.0, -80)])
def test_values_and_scores_far_from_one(level, size, S, bias):
    """V of size 2^size, scores around `level`: the weights are relative to the row's other weights, whatever the
    unit they are counted in, and so is out to V. Key and query share a RoPE value whose product bf16 operands
    and an fp32 sum hold exactly; the other scores are of size 1 (see TOL)."""
    x, _ = inputs(1, 150, S, 2, DSV3, torch.bfloat16, 81)
    x["k_rope"][..., 0] = 16.0
    x["q"][..., DSV3[1]] = level * 192 ** 0.5 / 16
    x["W_UV"] *= 2.0 ** size
    lo, hi = random_bounds(1, 150, S, 5)
    forward(x, lo, hi, **(dict(slopes=slopes(2)) if bias else {}))


@pytest.mark.parametrize("S", [300, 8300])
def test_scores_that_climb_and_fall(S):
    """Scores that rise or fall by 83 (2^120 in weight) every 40 keys, in steps that bf16 and fp32 hold exactly,
    and lie within a few units inside a step: the reference of a row's weights moves inside and between tiles."""
    x, _ = inputs(1, 200, S, 2, DSV3, torch.bfloat16, 82)
    x["k_rope"][0, :, 0] = (torch.arange(S, device=dev()) // 40 % 8).to(torch.bfloat16)
    q = torch.tensor([1152.0, -1152.0, 0.0, 64.0, -64.0], device=dev())
    x["q"][..., DSV3[1]] = q[torch.arange(400, device=dev()) % 5].view(1, 200, 2).to(torch.bfloat16)
    lo, hi = random_bounds(1, 200, S, 6)
    forward(x, lo, hi)


@pytest.mark.parametrize("dims", [(32, 160, 32, 200), (40, 200, 56, 256)])
def test_wide_heads_on_many_row_tiles_f32(dims):
    """Widths above 128 with enough row tiles for the CUDA-core forward's four rows a thread; rows that see
    nothing, so that the parts that a cluster's CTAs merge are empty for some."""
    x, dout = inputs(1, 520, 520, 8, dims, torch.float32, 83)
    lo, hi = random_bounds(1, 520, 520, 9)
    check(x, dout, key_lo=lo, key_hi=hi, causal=False, softcap=8.0, slopes=slopes(8))
