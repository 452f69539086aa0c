"""Masked attention where scores and values lie far from 1."""
import pytest
import torch

import masked_reference as ref
from mla_attention_sequence_gb300 import laga

from test_masked_gpu import DSV3, TOL, built, dev, inputs, random_bounds, slopes  # noqa: F401

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
