"""The plain forward on rows whose every score is far below zero: a softmax does not see a constant that is
added to all scores of a row, so neither out nor the row's weights may."""
import pytest
import torch

import masked_reference as ref
from mla_attention_sequence_gb300 import laga

from test_masked_gpu import DSV3, TOL, built, dev, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", ["materialize", "fused_recon", "simt"])
@pytest.mark.parametrize("level", [-200.0, -90.0, 200.0])
def test_scores_far_from_zero(variant, level):
    """The first RoPE value of every key is 8, so a query's first RoPE value moves all its scores by the same,
    through a product that bf16 operands and an fp32 sum hold exactly. The other scores are of size 1: out
    carries the roundings counted in TOL. lse: K's rounding, and 2^-24 of the raw product's 2800."""
    B, S, n_h = 1, 333, 2
    x, _ = inputs(B, S, S, n_h, DSV3, torch.bfloat16, 61)
    x["k_rope"][..., 0] = 8.0
    x["q"][:, ::2, :, DSV3[1]] = level * 192 ** 0.5 / 8
    out, lse = laga.fwd(*x.values(), variant=variant)
    want = ref.attention(x, ref.visible(S, S))
    ref.close({"out": out}, want, TOL[torch.bfloat16], ("out",))
    assert float((lse.double() - want["lse"]).abs().max()) <= 5e-2
    laga.check(dev())
