"""The 4-bit bounds of tests/q4_ref.py are as tight as they have to be: outputs
computed from the definition pass, and outputs of a kernel with a mistake (a code
bit lost, a warp's share of rows without their codes, one row too many, a token's
mask off by one) do not, at the long lengths too."""
import math

import pytest
import torch

from tests import cache_ref as ref, q4_ref

CASES = [([1152], 1, 4, 128), ([5000], 1, 3, 128), ([9001], 4, 4, 64), ([8200, 3], 1, 5, 128),
         ([300, 77], 2, 3, 64)]


def _rows(lens, H, d, g):
    out = []
    for n in lens:
        x = torch.randn(H, n, d, generator=g, dtype=torch.float64).to(torch.bfloat16).double()
        c, s, lo = ref.quantise(x)
        out.append((c, s, lo))
    return out


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"n{max(c[0])}T{c[1]}G{c[2]}d{c[3]}")
def test_bounds_see_mistakes(case):
    lens, T, G, d = case
    g = torch.Generator().manual_seed(d + T)
    K, V = _rows(lens, 1, d, g), _rows(lens, 1, d, g)
    q = (1.5 * torch.randn(len(lens), T, G, d, generator=g)).to(torch.bfloat16)
    scale = 1 / math.sqrt(d)
    e, lse, b, lb = q4_ref.attention(q, K, V, lens, scale)
    assert ((e.to(torch.bfloat16).double() - e).abs() <= b).all()

    def worst(V2=V, q2=q, lens2=lens):
        return float(((q4_ref.attention(q2, K, V2, lens2, scale)[0] - e).abs() / b).max())
    bit = [(torch.floor(c / 2) * 2, s, lo) for c, s, lo in V]
    assert worst(bit) > 2
    few = []  # every 8th row without its codes
    for c, s, lo in V:
        c = c.clone()
        c[:, ::8] = 8
        few.append((c, s, lo))
    assert worst(few) > 2
    share = []  # every second stage of 32 rows of a warp without its codes
    for c, s, lo in V:
        c = c.clone()
        for r in range(0, c.shape[1], 256):
            c[:, r:r + 32] = 8
        share.append((c, s, lo))
    assert worst(share) > 2
    lows = [(c, s, torch.zeros_like(lo)) for c, s, lo in V]
    assert worst(lows) > 2
    if max(lens) <= 1200:
        assert worst(lens2=[max(n - 1, 0) for n in lens]) > 1
