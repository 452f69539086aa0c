"""The training step that the README shows, run as it stands."""
import os
import re

import pytest
import torch

import masked_reference as ref
from mla_attention_sequence_gb300 import laga

from test_masked_gpu import DSV3, GRADS, TOL, built, dev, inputs, slopes  # noqa: F401

pytestmark = pytest.mark.gpu


def test_packed_training_step_with_checkpoints():
    """With queries of size 8 the scores are as large as a trained model's. The gradients are those of the
    attention that the forward computed: its weights sum to 1 in the backward too, and what is left of the
    checkpoints' error is that of D = rowsum(dout o out), half a step of e4m3 (2^-4) on out, which moves a
    gradient by at most as much of its uncancelled size, in the root mean square over sqrt(3); doubled for the
    roundings to bf16, which act on the weights in proportion to the scores."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        block, = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    B, S, n_h = 2, 300, 4
    x, dout = inputs(B, S, S, n_h, DSV3, torch.bfloat16, 91)
    x["q"] *= 8
    starts = [[0, 77, 290], [0, 128, 300]]
    g = torch.Generator().manual_seed(4)
    ns = dict(x, S=S, dout=dout, slopes=slopes(n_h) / 16,
              pos=torch.randint(0, 5000, (3, B, S), generator=g, dtype=torch.int32).to(dev()),
              doc_starts=torch.tensor(starts, dtype=torch.int32, device=dev()))
    exec(block, ns)  # leaves q and k_rope as the attention had them
    laga.check(dev())
    lo, hi = ref.bounds(starts, S, S)
    seen = ref.visible(S, S, torch.from_numpy(lo), torch.from_numpy(hi), B=B)
    y = {k: ns[k] for k in x}
    want = ref.attention(y, seen, 30.0, ns["slopes"], pos=torch.arange(S), dout=dout)
    # the scores' size times the rounding of K
    ref.close({"out": ns["out"]}, want, 8 * TOL[torch.bfloat16], ("out",))
    ref.close(ns["g"], want, 2 * 2.0 ** -4 / 3 ** 0.5, GRADS)
    assert ns["dq"].shape == x["q"].shape and ns["dk_rope"].shape == x["k_rope"].shape
