"""bf16 attention beside fp32 sums: with up to 16 queries a KV head the
probabilities reach V as two bf16 parts, so that what is left beside the output's
own rounding is 2^-16 of sum P |v| and fp32 sums."""
import math

import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from tests import cache_ref as ref
from tests.test_gpu_cache import BF, DEV, make_cache, rnd

pytestmark = pytest.mark.gpu

CASES = [
    # lens, n_new, H, G, d, bs
    ([1], 1, 1, 1, 64, 1),
    ([15, 16, 17, 127], 1, 1, 4, 128, 16),
    ([1152], 1, 8, 4, 128, 16),
    ([700, 1025, 64], 1, 3, 5, 128, 128),
    ([333, 40], 1, 2, 16, 128, 64),
    ([333, 1, 40], 1, 1, 16, 64, 256),
    ([3, 0, 1, 257], 3, 1, 5, 128, 8),
    ([9001], 4, 1, 4, 64, 16),
    ([8200, 3], 8, 2, 2, 128, 128),
]


@pytest.mark.parametrize("hidden", [False, True], ids=["", "nan"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"n{max(c[0])}T{c[1]}H{c[2]}G{c[3]}d{c[4]}")
def test_probabilities_in_two_parts(case, hidden):
    lens, T, H, G, d, bs = case
    S = len(lens)
    cache, table, rows = make_cache(S, H, d, bs, lens, "bf16", 17 + d)
    if hidden and T > 1:  # the newest row, a NaN to the last token alone
        for s in range(S):
            if lens[s]:
                cache[1][int(table[s, (lens[s] - 1) // bs]), :, (lens[s] - 1) % bs] = float("nan")
    q = rnd((S, T, H * G, d), BF, 3, scale=1.5)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = pkg.rkv_paged_attention(q, *cache, table, lens_d, lse=True)
    scale = 1 / math.sqrt(d)
    e, el, A, L = ref.attention(q, rows[0], rows[1], lens, scale)
    n = max(max(lens), 1)
    delta = L * (d + 4) * ref.U32 * scale + (el.abs().nan_to_num(0, 0, 0) + 8) * 4 * ref.U32
    b = (2 * delta[..., None] + (n / 2 + 128) * ref.U32 + 2.0 ** -16) * A
    b = b + ref.U16 * (e.abs() + b) + 1e-30
    err = (out.double().cpu() - e).abs() / b
    if hidden and T > 1:
        err = err[:, :-1]
    assert err.nan_to_num(9.0).max() <= 1, float(err.max())
