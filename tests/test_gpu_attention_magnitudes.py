"""Attention with logits of any size that fp32 holds: past 2^24 of them the spacing
of fp32 is wider than 1, and the weights of the largest must come out all the
same.  The products are whole numbers times powers of two, so that the logits are
exact and no two are closer than 2^-7 of themselves."""
import math

import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv
from tests import cache_ref as ref
from tests.test_gpu_cache import BF, DEV, FP, attend, gen, make_cache, rnd

pytestmark = pytest.mark.gpu

CASES = [([37], 1, 2, 64, 16), ([300, 5], 1, 4, 128, 16), ([1152], 1, 16, 128, 16), ([400], 8, 4, 64, 16),
         ([700, 1], 3, 2, 128, 64), ([9001], 1, 3, 64, 16), ([4000, 64, 3000] * 3, 2, 4, 128, 16)]


def whole_keys(cache, table, lens, kind, g):
    """Keys whose first element is a whole number of -60 .. 60 and the others 0; their
    values as fp64 rows [n] per sequence."""
    bs = (cache.shape if kind == "q4" else cache[0].shape)[2]
    if kind == "q4":
        cache.K_codes.zero_()
        cache.K_scales.zero_()
    else:
        cache[0].zero_()
    out = []
    for s, n in enumerate(lens):
        v = torch.randint(-60, 61, (n,), generator=g)
        for r in range(n):
            b = int(table[s, r // bs])
            if kind == "q4":
                cache.K_scales[b, :, r % bs, 0, 1] = float(v[r])  # the low of a group of zeros
            else:
                cache[0][b, :, r % bs, 0] = float(v[r])
        out.append(v.double())
    return out


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"S{len(c[0])}n{max(c[0])}T{c[1]}G{c[2]}d{c[3]}")
def test_logits_of_any_size(case, kind):
    lens, T, G, d, bs = case
    cache, table, rows = make_cache(len(lens), 1, d, bs, lens, kind, 60 + d, junk=False)
    keys = whole_keys(cache, table.cpu(), lens, kind, gen(d))
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for k in (0, 8, 15, 18, 20, 22, 25, 30, 33, 40, 60, 90, 110):
        q = torch.zeros(len(lens), T, G, d, dtype=FP if kind == "fp32" else BF, device=DEV)
        # each head its own factor and sign; one ordinary head among the large ones
        f = torch.tensor([(1.0, -0.75, 1.25, 2.0 ** -k)[i % 4] for i in range(G)], dtype=torch.float64)
        q[..., 0] = (f * 2.0 ** k).to(q.dtype).to(DEV)
        ws = pkg.alloc_attention_workspace(q, 1, max(lens))
        out, lse = attend(kind, q, cache, table, lens_d, max_rows=max(lens), scale=0.3, lse=True, workspace=ws)
        assert rkv.rkv_get_device_status(ws) == 0
        scale = float(torch.tensor(0.3, dtype=FP))
        for s, n in enumerate(lens):
            for t in range(T):
                see = n - T + t + 1
                if see <= 0:
                    assert (out[s, t] == 0).all()
                    continue
                z = (f * 2.0 ** k)[:, None] * keys[s][None, :see] * scale
                le = torch.logsumexp(z, -1)
                P = torch.softmax(z, -1)  # (le itself has 2^-53 of 2^100)
                v = rows[1][s][0, :see]
                e, A = P @ v, P @ v.abs()
                # a logit is off by 8 * 2^-24 of itself: what lies within 60 * 2^-24 of 60 of
                # the largest keeps its weight's order, the whole numbers are 1 apart
                far = torch.clamp(z.abs().amax(-1) * 8 * ref.U32, max=1.0) * (P.amax(-1) < 0.999)
                top = torch.exp((z - z.amax(-1, keepdim=True)).clamp(min=-700)).sum(-1)
                same = (z == z.amax(-1, keepdim=True)).sum(-1)
                sure = (top - same) < 1e-9  # the largest alone (with its equals) count
                delta = torch.where(sure, torch.zeros_like(far), far) + 40 * ref.U32
                b = (2 * delta[:, None] + (see / 2 + 128) * ref.U32) * A
                b = b + (2.0 ** -23 if kind == "fp32" else 2.0 ** -11 if kind == "q4" and T * G <= 16 else ref.U16) * \
                    (A + (v.abs().amax() if kind == "q4" else 0))
                b = b + (ref.U32 if kind == "fp32" else ref.U16) * (e.abs() + b)
                got = out[s, t].double().cpu()
                assert torch.isfinite(got).all(), (k, s, t)
                assert ((got - e).abs() <= b).all(), (k, s, t, float(((got - e).abs() / b).max()))
                assert ((lse[s, t].double().cpu() - le).abs() <= 16 * ref.U32 * (1 + le.abs()) + see * ref.U32).all()


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
def test_an_ordinary_query_beside_a_large_one(kind):
    """The same bits, whatever the size of the other queries of the call."""
    lens, T, G, d, bs = [500, 37], 2, 4, 128, 16
    cache, table, _ = make_cache(2, 1, d, bs, lens, kind, 70)
    q = rnd((2, T, G, d), FP if kind == "fp32" else BF, 3)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    a = attend(kind, q, cache, table, lens_d, max_rows=500)
    for k in (24, 60):
        big = q.clone()
        big[:, :, 1] *= 2.0 ** k
        b = attend(kind, big, cache, table, lens_d, max_rows=500)
        keep = [0, 2, 3]
        if kind == "q4":
            assert torch.equal(a[:, :, keep], b[:, :, keep])
        else:  # (a shared rescaling may move a sum's last bits)
            assert ((a[:, :, keep] - b[:, :, keep]).abs() <= 2.0 ** (-7 if kind == "bf16" else -18) * (a[:, :, keep].abs() + 0.1)).all()
        assert torch.isfinite(b).all()


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
@pytest.mark.parametrize("lens", [[1345], [357] * 20, [9001, 60]], ids=lambda n: f"S{len(n)}n{max(n)}")
def test_any_keys_and_large_queries(lens, kind):
    """Ordinary keys: one row has the weight where its logit is ahead of the others by
    more than fp32 may be off; everything is finite."""
    T, G, d, bs = 3, 2, 128, 16
    cache, table, rows = make_cache(len(lens), 1, d, bs, lens, kind, 5, junk=False)
    q0 = rnd((len(lens), T, G, d), FP if kind == "fp32" else BF, 7)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    scale = d ** -0.5
    for k in (3, 8, 14, 17, 20, 27, 33, 40, 60):
        q = q0 * 2.0 ** k
        out, lse = attend(kind, q, cache, table, lens_d, max_rows=max(lens), lse=True)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        for s, n in enumerate(lens):
            for t in range(T):
                kk, vv = (x[s][0, :n - T + t + 1] for x in rows)
                z = q[s, t].double().cpu() @ kk.T * scale
                two, at = z.topk(2, -1)
                # a logit is off by (d + 40) 2^-24 of sum |q| |k| at most (4 bits: of the groups'
                # parts, below 16 times that)
                off = (q[s, t].double().cpu().abs() @ kk.abs().T).amax(-1) * scale * (d + 40) * ref.U32 * 16
                for g in range(G):
                    if two[g, 0] - two[g, 1] > 2 * off[g] + 40:  # the others below e^-40
                        e = vv[at[g, 0]]
                        got = out[s, t, g].double().cpu()
                        # p = 1: the output's rounding, 4 bits also that of one product of the code
                        assert ((got - e).abs() <= 2.0 ** -7 * e.abs() + 2.0 ** -9 * vv.abs().amax()).all()
                assert ((lse[s, t].double().cpu() - torch.logsumexp(z, -1)).abs() <= off + 1e-4 + 2.0 ** -20 * z.abs().amax(-1)).all()
