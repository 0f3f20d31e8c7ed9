"""The 4-bit rows as the header states them, bit for bit: low, scale, and the
whole number nearest to t(x) * r with t(x) the fp32 nearest to x - low and r the
fp32 nearest to 1 / scale."""
import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from tests import cache_ref as ref
from tests.test_gpu_cache import BF, DEV, FP, gen

pytestmark = pytest.mark.gpu


def stated(x):
    """(codes, scale, low) of fp64 rows [..., d], with fp32 where it is stated."""
    g = x.unflatten(-1, (-1, 32))
    low = ref.floor_bf16(g.min(-1).values)
    # t of the largest, its fifteenth in fp32, then up to bf16
    t = (g.max(-1).values - low).float()
    scale = -ref.floor_bf16(-(t / 15).double())
    one = torch.ones_like(scale)
    r = torch.where(scale >= 2.0 ** -126, 1 / torch.where(scale > 0, scale, one), 0 * one).float().double()
    d = (g - low[..., None]).float().double()
    return torch.round(d * r[..., None]), scale, low


def written(x):
    """(codes, scale, low) of rows x [n, 1, d] in a cache, and read back."""
    n, _, d = x.shape
    c = pkg.alloc_q4_cache(n, 1, 1, d)
    table = torch.arange(n, dtype=torch.int32, device=DEV).view(n, 1)
    lens = torch.ones(n, dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    pkg.rkv_q4_append(c, xd, xd, table, lens)
    got = ref.unpack(c.K_codes.cpu()[:, 0, 0], c.K_scales.cpu()[:, 0, 0])
    again = ref.unpack(c.V_codes.cpu()[:, 0, 0], c.V_scales.cpu()[:, 0, 0])
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_as_stated(dt, d):
    g = gen(d)
    n = 4000
    x = torch.randn(n, 1, d, generator=g)
    x[::4] *= torch.exp2(torch.randint(-40, 1, (n // 4, 1, d), generator=g).float())  # far apart
    x[1::4] = torch.randint(-60, 60, (n // 4, 1, d), generator=g).float() / 8           # borders
    x[2::4] += 100.0
    # a group of -1.25, 6.25 and 2^-30: scale 0.5, and 2.5 + 2^-29 between two codes
    x[0, 0, :32] = torch.tensor([-1.25, 6.25] + [2.0 ** -30] * 30)
    x[1, 0, :32] = torch.tensor([-1.25, 6.25] + [-2.0 ** -30] * 30)
    # -2^-30 .. 7.5: t is 7.5, the scale 0.5
    x[2, 0, :32] = torch.tensor([-2.0 ** -30, 7.5] + [2.0] * 30)
    x = x.to(dt)
    code, scale, low = written(x)
    ec, es, el = stated(x[:, 0].double())
    assert torch.equal(low, el) and torch.equal(scale, es)
    assert torch.equal(code, ec)
    assert code[0, 0, 2] == 2 and scale[2, 0] == 0.5 and code.max() == 15 and code.min() == 0
