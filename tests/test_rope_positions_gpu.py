"""Rotation at positions as far as its stated bound reaches, against decimal arithmetic of 60 digits."""
from decimal import Decimal, getcontext

import math
import pytest
import torch

from mla_attention_sequence_gb300 import laga

from test_masked_gpu import built, dev  # noqa: F401

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.283185307179586476925286766559005768394338798750211641949889")


def turns(pos, theta, i, n):
    """pos * theta^(-i / n) in turns, modulo one, in [0, 1)."""
    getcontext().prec = 60
    t = Decimal(pos) * (-Decimal(i) / Decimal(n) * Decimal(theta).ln()).exp() / TWO_PI
    return float(t - t.to_integral_value(rounding="ROUND_FLOOR"))


@pytest.mark.parametrize("theta", [1.0, 100.0, 10000.0, 5e5, 1234567.891])
@pytest.mark.parametrize("d_rope", [2, 10, 64, 256])
def test_far_positions(theta, d_rope):
    """The angle is off by at most 2^-32 + |pos| 2^-65 turns, its fp32 value by 2^-26 more; then 2^-24 of the
    sine, the cosine, the products and their sum, as near positions have."""
    where = [0, 1, -1, 2 ** 23 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 33 + 7, 2 ** 40 + 3, -2 ** 44 - 11]
    n = d_rope // 2
    g = torch.Generator(device=dev()).manual_seed(3)
    k = torch.randn(1, len(where), d_rope, generator=g, device=dev())
    q = torch.randn(1, len(where), 1, d_rope, generator=g, device=dev())
    _, got = laga.rope(q, k, torch.tensor(where, device=dev()).view(1, 1, -1), theta=theta, interleaved=False)
    x = k[0].double().cpu()
    for r, p in enumerate(where):
        a = torch.tensor([2 * math.pi * turns(p, theta, i, n) for i in range(n)], dtype=torch.float64)
        u, v = x[r, :n], x[r, n:]
        want = torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()])
        size = float(x[r].abs().max()) * 2 ** 0.5
        off = 2 * math.pi * (2.0 ** -32 + abs(p) * 2.0 ** -65 + 2.0 ** -26)
        assert float((got[0, r].double().cpu() - want).abs().max()) <= (off + 8 * 2.0 ** -24) * size, p
