"""The 8-bit cache on the GPU: rows written and read back against 64-bit forms,
attention over them, both in a run with the compression, hidden and broken rows."""
import math

import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv
from tests import cache_ref as ref
from tests import q8_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rnd(shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(dtype).to(DEV)


def status(ws):
    return rkv.rkv_get_device_status(ws)


def tables(S, rows, bs, seed, extra=2):
    nb = max(1, -(-rows // bs))
    perm = torch.randperm(S * nb + extra, generator=gen(seed))[: S * nb]
    return perm.view(S, nb).to(torch.int32), S * nb + extra


# ------------------------------------------------------------------ append --

CASES = [
    # tokens of each sequence, older rows, heads, G, d, block, dtype, rot, interleaved
    ([1], [0], 1, 1, 64, 8, BF, 0, False),
    ([1, 1, 1], [5, 0, 130], 2, 3, 128, 16, BF, 128, False),
    ([7, 0, 33, 1], [3, 9, 0, 17], 8, 4, 128, 16, BF, 64, True),
    ([40, 2], [0, 64], 3, 1, 64, 1, FP, 64, False),
    ([5, 6, 7], [0, 1, 2], 5, 2, 128, 64, FP, 100, False),
    ([129, 300], [100, 0], 1, 2, 64, 128, BF, 32, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}-{c[2]}x{c[4]}-b{c[5]}-{str(c[6])[6:]}-r{c[7]}")
def test_append_and_read(case):
    counts, old, H, G, d, bs, dt, rot, inter = case
    S, total = len(counts), sum(counts)
    lens = [o + c for o, c in zip(old, counts)]
    table, nb = tables(S, max(lens), bs, 3)
    qkv = rnd((total, (G + 2) * H * d), dt, 11)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([G * H * d, H * d, H * d], -1))
    k[:, 0] *= 40.0
    v[0, 0, 5] = 0.0
    if total > 2:
        v[1, -1] = 0.0                      # a row of zeros
        v[2, 0] = 2.0 ** -140 if dt == FP else 2.0 ** -130  # below what a scale holds
    pos = torch.randint(0, 70000, (total,), generator=gen(4), dtype=torch.int32)
    cache = pkg.alloc_q8_cache(nb, H, bs, d)
    for t in (cache.K_codes, cache.V_codes):
        t.fill_(77)
    for t in (cache.K_scales, cache.V_scales):
        t.fill_(3.0)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    cu = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    plan = pkg.RopePlan(rot, interleaved=inter) if rot else None
    kw = dict(rope=plan, positions=pos.to(DEV)) if rot else {}
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    oq = pkg.rkv_q8_append(cache, k, v, table.to(DEV), lt, cu_tokens=cu.to(DEV), q=q, workspace=ws, **kw)
    assert status(ws) == 0
    f = ref.freqs(rot) if rot else torch.zeros(0, dtype=torch.float64)
    eq, ek = ref.rotate(q, pos, f, inter), ref.rotate(k, pos, f, inter)
    assert ((oq.double().cpu() - eq).abs() <= ref.rotate_bound(q, eq, rot, inter, dt)).all() if rot else torch.equal(oq, q)
    written = torch.zeros(nb, bs, dtype=torch.bool)
    codes, scales = q8_ref.quantise(v.double().cpu())
    at = 0
    for s in range(S):
        for i in range(counts[s]):
            r = old[s] + i
            b, o = int(table[s, r // bs]), r % bs
            written[b, o] = True
            assert torch.equal(cache.V_codes[b, :, o].cpu(), codes[at])
            assert torch.equal(cache.V_scales[b, :, o].cpu(), scales[at])
            kc, ks = cache.K_codes[b, :, o].cpu(), cache.K_scales[b, :, o].cpu()
            if not rot:
                ec, es = q8_ref.quantise(ek[at])
                assert torch.equal(kc, ec) and torch.equal(ks, es)
            else:
                # the turned row in fp32, then half a step and the scale's and the product's roundings
                lim = ref.rotate_bound(k[at: at + 1], ek[at: at + 1], rot, inter, FP)[0]
                got = kc.double() * ks.double()[:, None]
                big = ek[at].abs().amax(-1, keepdim=True)
                assert ((got - ek[at]).abs() <= lim + big / 127 * 0.5 * (1 + 2.0 ** -15) + big * 2.0 ** -22).all()
                assert ((ks.double() * 127 - big[:, 0]).abs() <= lim.amax(-1) + big[:, 0] * 2.0 ** -23).all()
            at += 1
    for c, s in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales)):
        rest = ~written
        assert (c.cpu().transpose(1, 2)[rest] == 77).all() and (s.cpu().transpose(1, 2)[rest] == 3.0).all()
    # read back: from row 0, and the new rows alone, in both types
    for first, n in ((None, max(lens)), ([o for o in old], max(counts))):
        for out in (BF, FP):
            ft = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
            oK = torch.full((S * H, n, d), 9.0, dtype=out, device=DEV)
            oV = torch.full_like(oK, 9.0)
            pkg.rkv_q8_read(cache, table.to(DEV), lt, n, first=ft, out_K=oK, out_V=oV, workspace=ws)
            for got, c, sc in ((oK, cache.K_codes, cache.K_scales), (oV, cache.V_codes, cache.V_scales)):
                want = torch.full_like(got, 9.0).cpu()
                for s in range(S):
                    for i in range(n):
                        r = i + (first[s] if first else 0)
                        if r < lens[s]:
                            b, o = int(table[s, r // bs]), r % bs
                            val = c[b, :, o].cpu().float() * sc[b, :, o].cpu()[:, None]  # (one rounding, as there)
                            want.view(S, H, n, d)[s, :, i] = val.to(out)
                assert torch.equal(got.cpu(), want)
    assert status(ws) == 0


def test_one_token_each_and_several():
    """Without cu_tokens: the same number of tokens each, from [S, n, H, d]."""
    S, n, H, d, bs = 5, 3, 4, 128, 16
    table, nb = tables(S, 40, bs, 8)
    lens = torch.tensor([3, 16, 17, 40, 9], dtype=torch.int32)
    k, v = rnd((S, n, H, d), BF, 1), rnd((S, n, H, d), BF, 2)
    a, b = (pkg.alloc_q8_cache(nb, H, bs, d) for _ in range(2))
    pkg.rkv_q8_append(a, k, v, table.to(DEV), lens.to(DEV))
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV) * n
    pkg.rkv_q8_append(b, k.flatten(0, 1), v.flatten(0, 1), table.to(DEV), lens.to(DEV), cu_tokens=cu)
    for x in ("K_codes", "K_scales", "V_codes", "V_scales"):
        assert torch.equal(getattr(a, x), getattr(b, x))
    assert (a.K_scales != 0).sum() == S * n * H


def test_rows_that_are_not_finite():
    """A NaN or an infinity: the row of that head reads as NaN, its neighbours as they are."""
    H, d, bs = 3, 64, 8
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([4], dtype=torch.int32, device=DEV)
    k, v = rnd((4, H, d), BF, 1), rnd((4, H, d), BF, 2)
    k[0, 1, 7], k[1, 0, 63], v[2, 2, 0] = math.nan, math.inf, -math.inf
    cache = pkg.alloc_q8_cache(1, H, bs, d)
    pkg.rkv_q8_append(cache, k, v, table, lens)
    K, V = pkg.rkv_q8_read(cache, table, lens, 4, dtype=FP)
    bad = torch.zeros(2, H, 4, dtype=torch.bool)
    bad[0, 1, 0] = bad[0, 0, 1] = bad[1, 2, 2] = True
    for i, got in enumerate((K, V)):
        assert torch.isnan(got.cpu()[bad[i]]).all() and torch.isfinite(got.cpu()[~bad[i]]).all()


def test_bad_rows_are_reported_and_skipped():
    H, d, bs = 2, 128, 16
    cache = pkg.alloc_q8_cache(2, H, bs, d)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    k, v = rnd((2, 1, H, d), BF, 1), rnd((2, 1, H, d), BF, 2)
    for table, lens in (([[0], [7]], [1, 1]), ([[0], [-1]], [1, 1]), ([[0], [1]], [1, 17]), ([[0], [1]], [1, 0])):
        for t in (cache.K_codes, cache.V_codes, cache.K_scales, cache.V_scales):
            t.zero_()
        table = torch.tensor(table, dtype=torch.int32, device=DEV)
        lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        pkg.rkv_q8_append(cache, k, v, table, lens, workspace=ws)
        assert status(ws) == 6 and status(ws) == 0
        assert (cache.V_scales != 0).sum() == H
        assert torch.equal(cache.V_codes[0, :, 0].cpu(), q8_ref.quantise(v[0, 0].double().cpu())[0])
    table = torch.tensor([[0], [9]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    pkg.rkv_q8_read(cache, table, lens, 1, workspace=ws)
    assert status(ws) == 6


# --------------------------------------------------------------- attention --

def make_cache(nb, H, bs, d, seed, spread=0.0):
    K, V = (torch.randn(nb, H, bs, d, generator=gen(seed + i)) for i in range(2))
    K += 0.5 * torch.randn(H, 1, d, generator=gen(seed + 2))
    if spread:
        V *= torch.exp2(spread * torch.randn(nb, H, bs, 1, generator=gen(seed + 3)))
    t = []
    for x in (K, V):
        c, s = q8_ref.quantise(x.double())
        t += [c.to(DEV), s.to(DEV)]
    return pkg.Q8Cache(*t)


def compare(q, cache, table, lens, out, lse, scale=None):
    S, T, hq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    rk = q8_ref.rows_of(cache.K_codes, cache.K_scales, table, lens)
    rv = q8_ref.rows_of(cache.V_codes, cache.V_scales, table, lens)
    e, el, A, L = ref.attention(q, rk, rv, lens, scale)
    b, bl = ref.attention_bounds(e, el, A, L, scale, d, max(max(lens), 1), "bf16")
    hidden = torch.isinf(el)
    assert torch.equal(torch.isinf(lse.cpu()), hidden)
    got = out.double().cpu()
    assert (got[hidden] == 0).all()
    assert ((got - e).abs() <= b).all(), float(((got - e).abs() / b).max())
    assert ((lse.double().cpu() - el).abs()[~hidden] <= bl[~hidden]).all()


ATTN = [
    # lens, n_new, H, G, d, block
    ([1], 1, 1, 1, 128, 16),
    ([1], 1, 1, 1, 64, 1),
    ([0, 1, 2, 31, 32, 33], 1, 2, 4, 128, 16),
    ([127, 128, 129, 500, 1152], 1, 8, 5, 128, 128),
    ([63, 64, 65, 200], 1, 3, 7, 64, 8),
    ([3, 2, 1, 0, 700], 5, 2, 3, 128, 32),       # tokens that see nothing
    ([777, 40, 64], 8, 2, 4, 64, 16),            # 32 queries
    ([260, 90], 2, 1, 8, 128, 64),               # 16 queries
    ([150, 9], 64, 1, 1, 64, 16),
    ([66, 300], 3, 1, 16, 128, 4),               # 48 queries
    ([9000], 1, 1, 2, 128, 16),                  # runs of the line, joined
    ([4000, 17, 2500, 3999] * 8, 1, 8, 4, 128, 128),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}-t{c[1]}-{c[2]}x{c[3]}x{c[4]}-b{c[5]}")
def test_attention(case):
    lens, T, H, G, d, bs = case
    S = len(lens)
    table, nb = tables(S, max(lens), bs, 5)
    cache = make_cache(nb, H, bs, d, 21)
    q = rnd((S, T, H * G, d), BF, 31)
    ws = pkg.alloc_attention_workspace(q, H, table.shape[1] * bs)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = pkg.rkv_q8_attention(q, cache, table.to(DEV), lt, lse=True, workspace=ws)
    assert status(ws) == 0
    compare(q, cache, table, lens, out, lse)
    again, _ = pkg.rkv_q8_attention(q, cache, table.to(DEV), lt, lse=True, workspace=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_attention_scales_and_sizes(scale):
    """Signs of the scale, values from row to row up to 2^30 apart, strided queries and outputs."""
    lens, T, H, G, d, bs = [130, 77], 2, 2, 4, 128, 16
    table, nb = tables(2, 130, bs, 6)
    cache = make_cache(nb, H, bs, d, 41, spread=8.0)
    big = rnd((2, T, H * G, 2 * d), BF, 51)
    q = big[..., d:]
    o = torch.zeros(2, H * G, T, d, dtype=BF, device=DEV).transpose(1, 2)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = pkg.rkv_q8_attention(q, cache, table.to(DEV), lt, scale=scale, out=o, lse=True)
    assert out.data_ptr() == o.data_ptr()
    compare(q, cache, table, lens, out, lse, scale)


def test_hidden_rows_may_hold_anything():
    """Rows past lens, and rows that only later tokens see: NaN scales and any codes there do not reach the
    others; the later tokens get NaN."""
    T, H, G, d, bs = 4, 1, 2, 64, 16
    lens = [50]
    table, nb = tables(1, 64, bs, 7)
    cache = make_cache(nb, H, bs, d, 61)
    q = rnd((1, T, H * G, d), BF, 71)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean, _ = pkg.rkv_q8_attention(q, cache, table.to(DEV), lt, lse=True)
    def at(r):
        return int(table[0, r // bs]), r % bs
    for r in range(50, 64):
        b, o = at(r)
        cache.K_scales[b, :, o] = math.nan
        cache.V_scales[b, :, o] = math.inf
        cache.V_codes[b, :, o] = -128
    assert torch.equal(pkg.rkv_q8_attention(q, cache, table.to(DEV), lt), clean)
    b, o = at(48)  # seen by tokens 2 and 3
    cache.V_scales[b, :, o] = math.nan
    out = pkg.rkv_q8_attention(q, cache, table.to(DEV), lt)
    assert torch.equal(out[:, :2], clean[:, :2]) and torch.isnan(out[:, 2:]).all()


def test_bad_ids_and_lengths():
    H, G, d, bs = 2, 2, 128, 16
    table, nb = tables(2, 64, bs, 9)
    cache = make_cache(nb, H, bs, d, 81)
    q = rnd((2, 1, H * G, d), BF, 91)
    ws = pkg.alloc_attention_workspace(q, H, 64)
    lt = torch.tensor([64, 40], dtype=torch.int32, device=DEV)
    t = table.clone()
    t[1, 1] = 99
    out, lse = pkg.rkv_q8_attention(q, cache, t.to(DEV), lt, lse=True, workspace=ws)
    assert status(ws) == 6
    rk = q8_ref.rows_of(cache.K_codes, cache.K_scales, table, [64, 40])
    rv = q8_ref.rows_of(cache.V_codes, cache.V_scales, table, [64, 40])
    keep = torch.ones(40, dtype=torch.bool)
    keep[16:32] = False
    rk[1], rv[1] = rk[1][:, keep], rv[1][:, keep]
    e, el, A, L = ref.attention(q, rk, rv, [64, 24], d ** -0.5)
    b, _ = ref.attention_bounds(e, el, A, L, d ** -0.5, d, 64, "bf16")
    assert ((out.double().cpu() - e).abs() <= b).all()
    long = torch.tensor([65, -3], dtype=torch.int32, device=DEV)
    out = pkg.rkv_q8_attention(q, cache, table.to(DEV), long, workspace=ws)
    assert status(ws) == 6 and (out[1] == 0).all() and torch.isfinite(out).all()


def test_captured_and_other_stream():
    """A step (append, attention) captured and replayed, and on a stream of its own: the bits of the calls."""
    S, H, G, d, bs = 3, 2, 4, 128, 16
    table, nb = tables(S, 200, bs, 10)
    lens = torch.tensor([200, 31, 97], dtype=torch.int32, device=DEV)
    q, k, v = rnd((S, 1, H * G, d), BF, 1), rnd((S, 1, H, d), BF, 2), rnd((S, 1, H, d), BF, 3)
    plan = pkg.RopePlan(d)
    tb = table.to(DEV)

    def step(cache, ws, out, oq):
        pkg.rkv_q8_append(cache, k, v, tb, lens, rope=plan, q=q, out_q=oq, workspace=ws)
        pkg.rkv_q8_attention(oq, cache, tb, lens, out=out, workspace=ws)
    res = []
    for kind in ("plain", "graph", "stream"):
        cache = make_cache(nb, H, bs, d, 33)
        ws = pkg.alloc_attention_workspace(q, H, tb.shape[1] * bs)
        out, oq = torch.zeros_like(q), torch.empty_like(q)
        torch.cuda.synchronize()
        if kind == "plain":
            step(cache, ws, out, oq)
        elif kind == "graph":
            step(cache, ws, out, oq)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(cache, ws, out, oq)
            out.zero_()
            g.replay()
        else:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step(cache, ws, out, oq)
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert status(ws) == 0
        res.append(out)
    assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


def test_run_with_the_compression():
    """Prompts written at 8 bits, read back, compressed, the kept rows written again, a decode step over them: the
    kept rows are those of the values read, and attention is that of the rows as stored."""
    S, H, G, d, bs, n, budget, n_obs = 2, 2, 4, 128, 16, 288, 192, 8
    table, nb = tables(S, n, bs, 12)
    k, v = rnd((S, n, H, d), BF, 1), rnd((S, n, H, d), BF, 2)
    cache = pkg.alloc_q8_cache(nb, H, bs, d)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    tb = table.to(DEV)
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    pkg.rkv_q8_append(cache, k, v, tb, lens, workspace=ws)
    K, V = pkg.rkv_q8_read(cache, tb, lens, n, workspace=ws)
    Q = rnd((S * H, G, n_obs, d), BF, 3)
    oK, oV, idx = pkg.rkv_compress(K, V, Q, n, budget, n_obs, 0.1, 2, 0.5)
    want = torch.gather(K, 1, idx.long()[..., None].expand(-1, -1, d))
    assert torch.equal(oK[:, :budget], want)
    kept = [x[:, :budget].reshape(S, H, budget, d).transpose(1, 2) for x in (oK, oV)]
    lens = torch.full((S,), budget, dtype=torch.int32, device=DEV)
    pkg.rkv_q8_append(cache, *kept, tb, lens, workspace=ws)
    new = [rnd((S, 1, H, d), BF, 5 + i) for i in range(2)]
    lens = lens + 1
    q = rnd((S, 1, H * G, d), BF, 9)
    pkg.rkv_q8_append(cache, *new, tb, lens, workspace=ws)
    out, lse = pkg.rkv_q8_attention(q, cache, tb, lens, lse=True)
    assert status(ws) == 0
    compare(q, cache, table, [budget + 1] * S, out, lse)


def test_python_refusals():
    c = pkg.alloc_q8_cache(2, 1, 8, 64)
    with pytest.raises(ValueError):
        pkg.Q8Cache(c.K_codes.to(torch.uint8), c.K_scales, c.V_codes, c.V_scales)
    with pytest.raises(ValueError):
        pkg.Q8Cache(c.K_codes, c.K_scales.to(BF), c.V_codes, c.V_scales)
    with pytest.raises(ValueError):
        pkg.Q8Cache(c.K_codes, c.K_scales, c.V_codes[:1], c.V_scales)
    with pytest.raises(ValueError):
        pkg.Q8Cache(c.K_codes.cpu(), c.K_scales, c.V_codes, c.V_scales)
    with pytest.raises(rkv.RkvError) as e:
        t = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
        pkg.rkv_q8_attention(rnd((1, 1, 1, 64), FP, 1), c, t, torch.ones(1, dtype=torch.int32, device=DEV))
    assert e.value.code == 2
