"""Shared prefixes and 8-bit caches in the last blocks of pools whose bytes and
elements pass 32 bits: the bits of the same rows in a small pool."""
import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
H, G, D, BS = 2, 4, 128, 16
FAR = (1 << 32) // (H * BS * D) + 40  # blocks: more than 2^32 elements
USED = 30


def rnd(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def room():
    need = 6 * FAR * H * BS * D * 4
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("the device's free memory does not hold the pools")
    yield
    torch.cuda.empty_cache()


def places():
    """Ids of the small pool's blocks in the large one, some near its beginning."""
    return [i if i % 5 == 0 else FAR - 1 - i for i in range(USED)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("seqs", [4, 40])
def test_prefixes_far_in_a_pool(seqs, dtype):
    at = torch.tensor(places())
    small = [rnd((USED, H, BS, D), dtype, 1 + i) for i in range(2)]
    large = [torch.empty(FAR, H, BS, D, dtype=dtype, device=DEV) for _ in range(2)]
    for x, y in zip(small, large):
        y[at.to(DEV)] = x
    table = torch.arange(USED, dtype=torch.int32)
    ptable, own = table[:20].view(1, 20), table[20:].repeat(4, 1).view(-1, 1)[:seqs]
    q = rnd((seqs, 1, H * G, D), dtype, 5)
    plens, lens = ints([20 * BS - 3]), ints([1 + i % BS for i in range(seqs)])
    ws = pkg.alloc_prefix_attention_workspace(q, H, BS, 1, 20 * BS)
    a, la = pkg.rkv_prefix_attention(q, *small, ptable.to(DEV), plens, own.to(DEV).contiguous(), lens, lse=True, workspace=ws)
    to = at.to(torch.int32)
    b, lb = pkg.rkv_prefix_attention(q, *large, to[ptable.long()].to(DEV), plens, to[own.long()].to(DEV), lens, lse=True,
                                     workspace=ws)
    assert rkv.rkv_get_device_status(ws) == 0
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.isfinite(b).all()


def test_eight_bits_far_in_a_pool():
    at = torch.tensor(places())
    small = pkg.alloc_q8_cache(USED, H, BS, D)
    large = pkg.Q8Cache(*[torch.empty(FAR, *x.shape[1:], dtype=x.dtype, device=DEV)
                          for x in (small.K_codes, small.K_scales, small.V_codes, small.V_scales)])
    table = torch.arange(USED, dtype=torch.int32).view(3, 10)
    lens, n = [160, 37, 100], 37
    k, v = (rnd((3, n, H, D), torch.bfloat16, 7 + i) for i in range(2))
    q = rnd((3, n, H * G, D), torch.bfloat16, 9)
    for x in (small.K_codes, small.K_scales, small.V_codes, small.V_scales):
        x.fill_(1)
    for x in ("K_codes", "K_scales", "V_codes", "V_scales"):
        getattr(large, x)[at.to(DEV)] = getattr(small, x)
    res = []
    for cache, t in ((small, table), (large, at.to(torch.int32)[table.long()])):
        t = t.to(DEV).contiguous()
        ws = pkg.alloc_attention_workspace(q, H, 160)
        turned = pkg.rkv_q8_append(cache, k, v, t, ints(lens), rope=pkg.RopePlan(D), q=q, workspace=ws)
        out = pkg.rkv_q8_attention(turned, cache, t, ints(lens), lse=True, workspace=ws)
        res.append([turned, *out, *pkg.rkv_q8_read(cache, t, ints(lens), 160, dtype=torch.float32, workspace=ws)])
        assert rkv.rkv_get_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*res)) and all(torch.isfinite(x).all() for x in (res[1][0], *res[1][3:]))
