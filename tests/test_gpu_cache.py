"""The cache in use on the GPU against plain 64-bit forms: rotary positions,
appends (paged, 4 bits), reading back, attention; and runs of them together
with the compression."""
import math

import numpy as np
import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv
from tests import cache_ref as ref

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


# ------------------------------------------------------------------ rotary --

ROPE_CASES = [
    # tokens, heads, kv heads, d, rot, interleaved, dtype, scaling
    (1, 1, 1, 64, 64, False, BF, {}),
    (7, 4, 2, 128, 128, False, BF, {}),
    (33, 5, 1, 128, 64, True, BF, dict(scaling="by_parts", factor=8.0, original_len=8192.0, high=4.0)),
    (130, 3, 3, 64, 2, False, FP, {}),
    (64, 32, 8, 128, 128, False, FP, dict(scaling="ntk", factor=4.0)),
    (19, 2, 1, 128, 100, False, BF, dict(scaling="linear", factor=3.0)),  # steps of one pair
    (19, 2, 1, 128, 100, True, FP, {}),
    (2049, 1, 1, 64, 32, False, BF, {}),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[3]}-{c[4]}-{c[5]}-{str(c[6])[6:]}")
def test_rope(case, inverse):
    n, hq, hk, d, rot, inter, dt, sc = case
    m = 1.0 if not sc else 1.25
    plan = pkg.RopePlan(rot, interleaved=inter, attn_factor=m, **sc)
    f = ref.freqs(rot, **sc)
    qkv = rnd((n, (hq + 2 * hk) * d), dt, n + d)  # slices of a fused projection
    q, k = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
    pos = torch.randint(-3, 131072, (n,), generator=gen(5), dtype=torch.int32)
    pos[0] = 2 ** 31 - 1 if rot <= 64 else 0
    before = qkv.clone()
    oq, ok = pkg.rkv_rope_apply(plan, pos.to(DEV), q, k, inverse=inverse)
    assert torch.equal(qkv, before)
    for x, y in ((q, oq), (k, ok)):
        e = ref.rotate(x, pos, f, inter, m, inverse)
        # position 2^31 - 1: the plan's own rounding counts, 2^-20.6 of a turn at most
        b = ref.rotate_bound(x, e, rot, inter, dt, m)
        far = (pos.abs() > 2 ** 27).double()[:, None, None] * 2.0 ** -17 * x.double().cpu().abs().amax()
        assert ((y.double().cpu() - e).abs() <= b + far).all()
    # in place, on the slices themselves: the same bits
    r = pkg.rkv_rope_apply(plan, pos.to(DEV), q, k, out_q=q, out_k=k, inverse=inverse)
    assert r[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


@pytest.mark.parametrize("order", ["sequence", "token"])
def test_rope_in_place_of_several_sequences(order):
    """Slices of a projection whose rows lie sequence by sequence or token by
    token, turned in place: the bits of a call with outputs of its own."""
    S, n, hq, hk, d = 3, 5, 4, 2, 64
    plan = pkg.RopePlan(d)
    qkv = rnd((S, n, (hq + 2 * hk) * d) if order == "sequence" else (n, S, (hq + 2 * hk) * d), BF, 77)
    rows = qkv if order == "sequence" else qkv.transpose(0, 1)
    q = rows[..., :hq * d].unflatten(-1, (hq, d))
    k = rows[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    pos = torch.arange(S * n, dtype=torch.int32, device=DEV)
    oq, ok = pkg.rkv_rope_apply(plan, pos, q.contiguous(), k.contiguous())
    v = rows[..., (hq + hk) * d:].clone()
    pkg.rkv_rope_apply(plan, pos, q, k, out_q=q, out_k=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(rows[..., (hq + hk) * d:], v)


def test_rope_is_the_gradients_map():
    """<R x, y> = <x, R^T y>, and R^T is the derivative: differences of the
    forward pass (linear, so any step is exact) along every input."""
    plan = pkg.RopePlan(64, interleaved=True, attn_factor=0.75)
    n, d = 5, 64
    pos = torch.tensor([0, 3, 900, 70000, 131071], dtype=torch.int32, device=DEV)
    x, y = rnd((n, 1, d), FP, 1), rnd((n, 1, d), FP, 2)
    fx = pkg.rkv_rope_apply(plan, pos, x)
    bty = pkg.rkv_rope_apply(plan, pos, y, inverse=True)
    a = (fx.double() * y.double()).sum((1, 2))
    b = (x.double() * bty.double()).sum((1, 2))
    # each side: d terms, each off by at most 8 * 2^-24 (|x| + |x'|) |y|
    lim = 16 * 2.0 ** -24 * 2 * (x.double().norm(dim=(1, 2)) * y.double().norm(dim=(1, 2))) * 2
    assert ((a - b).abs() <= lim).all()
    # the derivative of sum(y * R x) along each input, by a difference of step 1
    eye = torch.eye(d, device=DEV)[:, None, :].expand(d, n, d).reshape(d * n, 1, d).contiguous()
    moved = pkg.rkv_rope_apply(plan, pos.repeat(d), eye)
    grad = (moved.view(d, n, d).double() * y.view(1, n, d).double()).sum(-1).T
    assert ((grad - bty.view(n, d).double()).abs() <= 32 * 2.0 ** -24 * y.double().abs().amax()).all()


def test_rope_shapes_and_empty():
    plan = pkg.RopePlan(128)
    q = rnd((3, 4, 8, 128), BF, 9)
    pos = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)
    y = pkg.rkv_rope_apply(plan, pos, q)
    z = pkg.rkv_rope_apply(plan, pos.reshape(-1), q.view(12, 8, 128))
    assert torch.equal(y.view(12, 8, 128), z)
    # a transposed layout [heads, tokens, d], as the compression's Q_obs rows lie
    t = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(pkg.rkv_rope_apply(plan, pos, t), y)
    assert pkg.rkv_rope_apply(plan, pos[:0].reshape(-1), q.view(12, 8, 128)[:0]).shape == (0, 8, 128)
    # the caller's own angles
    own = pkg.RopePlan(128, freqs=ref.freqs(128).tolist())
    assert torch.equal(pkg.rkv_rope_apply(own, pos, q), y)


# ------------------------------------------------------------------ append --

def make_table(S, nb, extra, seed):
    perm = torch.randperm(S * nb + extra, generator=gen(seed))[:S * nb]
    t = torch.full((S, nb + 1), 1 << 30, dtype=torch.int32)  # past the blocks in use: no ids
    t[:, :nb] = perm.view(S, nb).to(torch.int32)
    return t


APPEND_CASES = [
    # seqs, H, G, d, bs, new (list: ragged), dtype, rot, interleaved
    (1, 1, 1, 64, 1, 1, BF, 64, False),
    (3, 2, 4, 128, 16, 1, BF, 128, False),
    (5, 8, 5, 128, 128, 3, FP, 64, True),
    (4, 3, 16, 64, 8, [0, 17, 1, 40], BF, 64, False),
    (2, 2, 2, 128, 32, [129, 70], FP, 100, False),
    (40, 1, 1, 64, 16, [i % 4 for i in range(40)], BF, 0, False),
    (3, 8, 4, 128, 16, [64, 0, 333], BF, 128, True),
]


def _append_inputs(case, seed=0):
    S, H, G, d, bs, new, dt, rot, inter = case
    counts = new if isinstance(new, list) else [new] * S
    total = sum(counts)
    rng = np.random.RandomState(seed + S)
    lens = [c + (int(rng.randint(0, 3 * bs + 5)) if c else int(rng.randint(0, 5))) for c in counts]
    nb = max(1, -(-max(lens) // bs))
    table = make_table(S, nb, 3, seed + 1)
    qkv = rnd((total, (G * H + 2 * H) * d), dt, seed + 2)
    q = qkv[:, :G * H * d].view(total, G * H, d)
    k = qkv[:, G * H * d:(G + 1) * H * d].view(total, H, d)
    v = qkv[:, (G + 1) * H * d:].view(total, H, d)
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    pos = torch.randint(0, 131072, (total,), generator=gen(seed + 3), dtype=torch.int32)
    return counts, lens, nb, table, q, k, v, cu, pos


def _slots(counts, lens, table, bs):
    blk, row = [], []
    for s, c in enumerate(counts):
        for r in range(lens[s] - c, lens[s]):
            blk.append(int(table[s, r // bs]))
            row.append(r % bs)
    return torch.tensor(blk, dtype=torch.long), torch.tensor(row, dtype=torch.long)


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: f"S{c[0]}H{c[1]}G{c[2]}d{c[3]}bs{c[4]}r{c[7]}")
def test_paged_append(case):
    S, H, G, d, bs, new, dt, rot, inter = case
    counts, lens, nb, table, q, k, v, cu, pos = _append_inputs(case)
    ragged = isinstance(new, list)
    plan = pkg.RopePlan(rot, interleaved=inter) if rot else None
    K = torch.full((S * nb + 3, H, bs, d), -7.5, dtype=dt, device=DEV)
    V = torch.full_like(K, 3.25)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = pkg.rkv_paged_append(K, V, k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                               cu_tokens=cu.to(DEV) if ragged else None, rope=plan,
                               positions=pos.to(DEV) if rot else None, q=q, workspace=ws)
    assert status(ws) == 0
    f = ref.freqs(rot) if rot else torch.zeros(0, dtype=torch.float64)
    blk, row = _slots(counts, lens, table, bs)
    eq = ref.rotate(q, pos, f, inter)
    assert ((out.double().cpu() - eq).abs() <= ref.rotate_bound(q, eq, rot, inter, dt)).all()
    if not rot:
        assert torch.equal(out, q)
    ek = ref.rotate(k, pos, f, inter)
    Kc, Vc = K.cpu(), V.cpu()
    assert ((Kc[blk, :, row].double() - ek).abs() <= ref.rotate_bound(k, ek, rot, inter, dt)).all()
    assert torch.equal(Vc[blk, :, row], v.cpu())
    Kc[blk, :, row], Vc[blk, :, row] = -7.5, 3.25  # nothing else has changed
    assert (Kc == -7.5).all() and (Vc == 3.25).all()


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: f"S{c[0]}H{c[1]}G{c[2]}d{c[3]}bs{c[4]}r{c[7]}")
def test_q4_append_and_read(case):
    S, H, G, d, bs, new, dt, rot, inter = case
    counts, lens, nb, table, q, k, v, cu, pos = _append_inputs(case, seed=50)
    ragged = isinstance(new, list)
    plan = pkg.RopePlan(rot, interleaved=inter) if rot else None
    c = pkg.alloc_q4_cache(S * nb + 3, H, bs, d)
    for t in (c.K_codes, c.V_codes):
        t.fill_(0xA5)
    for t in (c.K_scales, c.V_scales):
        t.fill_(-7.5)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = pkg.rkv_q4_append(c, k, v, table.to(DEV), lens_d, cu_tokens=cu.to(DEV) if ragged else None,
                            rope=plan, positions=pos.to(DEV) if rot else None, q=q, workspace=ws)
    assert status(ws) == 0
    f = ref.freqs(rot) if rot else torch.zeros(0, dtype=torch.float64)
    eq = ref.rotate(q, pos, f, inter)
    assert ((out.double().cpu() - eq).abs() <= ref.rotate_bound(q, eq, rot, inter, dt)).all()
    blk, row = _slots(counts, lens, table, bs)
    for codes, scales, x in ((c.K_codes, c.K_scales, ref.rotate(k, pos, f, inter)),
                             (c.V_codes, c.V_scales, v.double().cpu())):
        is_k = codes is c.K_codes
        code, s, lo = ref.unpack(codes.cpu()[blk, :, row], scales.cpu()[blk, :, row])
        back = (code * s[..., None] + lo[..., None]).flatten(-2)
        # half a step, the fp32 rounding of x - low and of the product (2^-23 of 15
        # steps), and the rotation's own error
        b = s.repeat_interleave(32, -1) * (0.5 + 2.0 ** -19)
        b = b + 2.0 ** -24 * (x.abs() + lo.abs().repeat_interleave(32, -1))
        if is_k:
            b = b + ref.rotate_bound(k, x, rot, inter, FP)
        assert ((back - x).abs() <= b).all()
        if not rot or not is_k:
            # no rotation: codes, scales and lows as defined, bit for bit, but where fp32
            # moves (x - low) * r across a border (x - low not exact and next to a half)
            ec, es, el = ref.quantise(x)
            assert torch.equal(s, es) and torch.equal(lo, el)
            y = (x.unflatten(-1, (-1, 32)) - lo[..., None]) / s[..., None].clamp(min=1e-300)
            near = ((y - y.floor()) - 0.5).abs() <= 15 * 2.0 ** -23
            exact = (x.unflatten(-1, (-1, 32)) - lo[..., None]).float().double() == \
                (x.unflatten(-1, (-1, 32)) - lo[..., None])
            assert ((code == ec) | (near & ~exact)).all()
    # reading back: the same values in bf16 and fp32, other rows left alone
    n_read = max(counts) + 2
    first = torch.tensor([n - m for n, m in zip(lens, counts)], dtype=torch.int32, device=DEV)
    for rd in (BF, FP):
        oK = torch.full((S * H, n_read, d), 9.0, dtype=rd, device=DEV)
        oV = torch.full_like(oK, 9.0)
        pkg.rkv_q4_read(c, table.to(DEV), lens_d, n_read, first=first, out_K=oK, out_V=oV, workspace=ws)
        assert status(ws) == 0
        for codes, scales, o in ((c.K_codes, c.K_scales, oK), (c.V_codes, c.V_scales, oV)):
            val = ref.values(codes.cpu()[blk, :, row], scales.cpu()[blk, :, row])
            exp = torch.full((S, H, n_read, d), 9.0, dtype=torch.float64)
            j = 0
            for s, n in enumerate(counts):
                exp[s, :, :n] = val[j:j + n].transpose(0, 1)
                j += n
            got = o.double().cpu().view(S, H, n_read, d)
            # scale * code + low in one fp32 rounding, then one to the output's type
            u = 2.0 ** -24 + (2.0 ** -8 if rd == BF else 0.0)
            assert ((got - exp).abs() <= u * 1.01 * exp.abs() + 1e-37).all()
    c.K_codes[blk.to(DEV), :, row.to(DEV)] = 0xA5
    c.V_scales[blk.to(DEV), :, row.to(DEV)] = -7.5
    assert (c.K_codes == 0xA5).all() and (c.V_scales == -7.5).all()  # nothing else has changed


def test_q4_groups_of_special_values():
    """Constant groups, zeros, halves between codes, the largest floats, NaN
    and infinities (the whole group reads as NaN, the others are untouched)."""
    d, rows = 128, 9
    x = torch.zeros(rows, 1, d)
    x[1] = 3.0                                   # representable constant
    x[2] = 1.0 + 2.0 ** -20                      # constant that bf16 does not hold
    x[3, 0, :32] = torch.arange(32) % 16 + 0.0   # every code
    x[3, 0, 32:64] = torch.arange(32) / 2.0 - 0.5  # steps of 1: halves go to even codes
    x[4, 0, 5] = float("nan")
    x[5, 0, 70] = float("inf")
    x[6, 0, :2] = torch.tensor([3e38, -3e38])    # a range past the largest float
    x[7, 0, 100] = 1e-40                         # a scale below 2^-126: the low value stays
    x[8, 0, :2] = torch.tensor([3e38, 1e38])
    c = pkg.alloc_q4_cache(rows, 1, 1, d)
    table = torch.arange(rows, dtype=torch.int32, device=DEV).view(rows, 1)
    lens = torch.ones(rows, dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    pkg.rkv_q4_append(c, xd, xd, table, lens)
    K, V = pkg.rkv_q4_read(c, table, lens, 1, dtype=FP)
    assert torch.equal(K.view(torch.int32), V.view(torch.int32))
    got, groups = K.view(rows, 4, 32).cpu().double(), x.view(rows, 4, 32).double()
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    bad[4, 0] = bad[5, 2] = bad[6, 0] = True
    assert torch.isnan(got[bad]).all() and not torch.isnan(got[~bad]).any()
    for r in (0, 1, 2, 3, 8):
        code, s, lo = ref.quantise(groups[r].reshape(1, -1))
        assert torch.allclose(got[r].reshape(-1), (code * s[..., None] + lo[..., None]).reshape(-1),
                              rtol=2.0 ** -23, atol=0)
    assert (got[7].abs() <= 1e-40).all() and (got[6, 1:] == 0).all()


def test_append_padding_and_bad_ids():
    """Tokens past cu_tokens[num_seqs] do nothing; rows outside the table and
    ids that name no block are recorded and skipped, everything else lands."""
    S, H, d, bs = 3, 2, 64, 8
    table = make_table(S, 2, 0, 1)
    table[1, 0] = 99
    K = torch.zeros(S * 2, H, bs, d, dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    k, v, q = rnd((20, H, d), BF, 1), rnd((20, H, d), BF, 2), rnd((20, 2 * H, d), BF, 3)
    cu = torch.tensor([0, 5, 6, 9], dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 3, 26], dtype=torch.int32, device=DEV)  # 26: past the table's 24 rows
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    oq = torch.full_like(q, 5.0)
    pkg.rkv_paged_append(K, V, k, v, table.to(DEV), lens, cu_tokens=cu, q=q, out_q=oq, workspace=ws)
    assert status(ws) == rkv.RKV_ERR_DEVICE and status(ws) == 0
    assert torch.equal(oq[:9], q[:9]) and (oq[9:] == 5.0).all()
    exp = torch.zeros_like(K).cpu()
    for j in range(5):
        exp[int(table[0, 0]), :, j] = k[j].cpu()
    # sequence 2: rows 23, 24, 25 of a table of 3 * 8 rows whose third block has no id
    assert torch.equal(K.cpu(), exp)
    c = pkg.alloc_q4_cache(S * 2, H, bs, d)
    pkg.rkv_q4_append(c, k, v, table.to(DEV), lens, cu_tokens=cu, workspace=ws)
    assert status(ws) == rkv.RKV_ERR_DEVICE
    assert int((c.K_scales.flatten(1).abs().sum(1) != 0).sum()) == 1  # one block written
    lens[2] = 1  # fewer rows than tokens: rows -2, -1 do not exist, row 0 is written
    pkg.rkv_paged_append(K, V, k, v, table.to(DEV), lens, cu_tokens=cu, workspace=ws)
    assert status(ws) == rkv.RKV_ERR_DEVICE
    assert torch.equal(K[int(table[2, 0]), :, 0], k[8])


def test_append_rows_of_a_compression():
    """The kept rows of rkv_compress ([P, rows, d], heads outside tokens) go to
    a 4-bit cache as they lie; positions default to the rows."""
    S, H, n, d = 2, 3, 40, 64
    kept = rnd((S * H, 64, d), BF, 4)
    view = kept.view(S, H, 64, d)[:, :, :n].transpose(1, 2)  # [S, n, H, d], strided
    table = torch.arange(S * 3, dtype=torch.int32, device=DEV).view(S, 3)
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    K = torch.zeros(S * 3, H, 16, d, dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    plan = pkg.RopePlan(64)
    pkg.rkv_paged_append(K, V, view, view, table, lens, rope=plan)
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    pkg.rkv_paged_append(K2, V2, view, view, table, lens, rope=plan,
                         positions=torch.arange(n, dtype=torch.int32, device=DEV).repeat(S))
    assert torch.equal(K, K2)
    got = V.view(S, 3, H, 16, d).transpose(1, 2).reshape(S, H, 48, d)[:, :, :n]
    assert torch.equal(got, kept.view(S, H, 64, d)[:, :, :n])


# --------------------------------------------------------------- attention --

def make_cache(S, H, d, bs, lens, kind, seed, extra=2, junk=True):
    """(pools or Q4Cache, table, fp64 rows per sequence).  Rows past the
    sequences and unused blocks hold NaN (junk)."""
    nb = max(1, -(-max(max(lens), 1) // bs))
    table = make_table(S, nb, extra, seed)
    blocks = S * nb + extra
    dt = FP if kind == "fp32" else BF
    shift = torch.randn(H, 1, d, generator=gen(seed + 7))
    K = torch.randn(blocks, H, bs, d, generator=gen(seed + 8)) + shift
    V = torch.randn(blocks, H, bs, d, generator=gen(seed + 9))
    keep = torch.zeros(blocks, bs, dtype=torch.bool)
    for s in range(S):
        for r in range(lens[s]):
            keep[int(table[s, r // bs]), r % bs] = True
        for b in range(-(-max(lens[s], 0) // bs), nb + 1):
            table[s, b] = -5 if b % 2 else 1 << 29  # never looked at
    if kind == "q4":
        arr = []
        for x in (K, V):
            c, sc, lo = ref.quantise(x.to(BF).double())
            W = d // 32
            h = c.to(torch.int64).unflatten(-1, (8, 4)).transpose(-3, -2)  # [.., 8, W, 4]
            b = torch.stack([h[..., 0] | h[..., 1] << 4, h[..., 2] | h[..., 3] << 4], -1)
            codes = b.flatten(-3).to(torch.uint8)
            scales = torch.stack([sc, lo], -1).to(BF)
            if junk:
                scales[~keep[:, None].expand(-1, H, -1)] = float("nan")
            arr += [codes.contiguous().to(DEV), scales.contiguous().to(DEV)]
            assert codes.shape[-1] == d // 2 and W == scales.shape[-2]
        cache = pkg.Q4Cache(*arr)
        kv = ref.values(cache.K_codes, cache.K_scales), ref.values(cache.V_codes, cache.V_scales)
    else:
        K, V = K.to(dt), V.to(dt)
        if junk:
            K[~keep[:, None].expand(-1, H, -1)] = float("nan")
            V[~keep[:, None].expand(-1, H, -1)] = float("inf")
        cache = (K.to(DEV), V.to(DEV))
        kv = K.double(), V.double()
    rows = []
    for x in kv:
        per = []
        for s in range(S):
            ids = table[s, :nb].long().clamp(0, blocks - 1)
            per.append(x[ids].transpose(0, 1).reshape(H, nb * bs, d)[:, :lens[s]])
        rows.append(per)
    return cache, table.to(DEV), rows


def attend(kind, q, cache, table, lens, **kw):
    if kind == "q4":
        return pkg.rkv_q4_attention(q, cache, table, lens, **kw)
    return pkg.rkv_paged_attention(q, cache[0], cache[1], table, lens, **kw)


def check_attention(kind, q, out, lse, rows, lens, scale, cache=None):
    d = q.shape[-1]
    e, el, A, L = ref.attention(q, rows[0], rows[1], lens, scale)
    extra = extra_v = 0.0
    if kind == "q4":
        # the constant 128 and the lows: sums of |q| times up to 143 scales and |low|, a few
        # roundings each; the same for the values, where the rounded p * scale meets codes 0 .. 15
        smax = max(float(cache.K_scales.nan_to_num(0)[..., 0].max()), 0)
        lmax = float(cache.K_scales.nan_to_num(0)[..., 1].abs().max())
        qs = float(q.double().abs().sum(-1).max())
        extra = qs * (143 * smax + lmax) * 8 * ref.U32
        sv = float(cache.V_scales.nan_to_num(0)[..., 0].max())
        lv = float(cache.V_scales.nan_to_num(0)[..., 1].abs().max())
        extra_v = ref.U16 * 15 * sv + (143 * sv + lv) * (max(lens) / 4 + 64) * ref.U32
    b, bl = ref.attention_bounds(e, el, A, L, scale, d, max(max(lens), 1), kind, extra, extra_v)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - e).abs() <= b).all(), float(((got - e).abs() / b).max())
    hidden = torch.isinf(el)
    assert torch.equal(hidden, torch.isinf(lse.cpu())) and (got[hidden] == 0).all()
    dl = (lse.double().cpu() - el).abs()[~hidden]
    assert (dl <= bl[~hidden]).all()


ATTN_CASES = [
    # lens, n_new, H, G, d, bs
    ([1], 1, 1, 1, 64, 1),
    ([0, 1, 2, 31], 1, 2, 1, 128, 8),
    ([15, 16, 17, 127], 1, 1, 4, 128, 16),
    ([129, 5, 0, 200], 1, 2, 8, 64, 32),
    ([1152], 1, 8, 4, 128, 16),
    ([700, 1025, 64], 1, 3, 5, 128, 128),
    ([333, 40], 1, 2, 16, 128, 64),
    ([333, 1, 40], 1, 1, 7, 64, 256),
    ([3, 8, 300, 65], 8, 2, 4, 64, 16),
    ([3, 0, 1, 257], 4, 1, 5, 128, 8),
    ([90, 20], 2, 2, 3, 128, 1),
    ([100, 70], 64, 1, 2, 64, 16),
    ([5000], 1, 1, 3, 128, 1024),
    ([4224, 17, 2048], 3, 1, 16, 64, 4),
    # long enough, or enough sequences, that pieces of them are joined by a second launch
    ([9001], 4, 1, 4, 64, 16),
    ([8200, 3], 1, 2, 5, 128, 128),
    ([(i * 37) % 300 for i in range(45)], 1, 1, 2, 64, 16),
    ([700, 1, 0, 650] * 10, 2, 1, 16, 128, 32),
    ([i % 7 * 40 for i in range(300)], 1, 1, 1, 64, 8),
]


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: f"S{len(c[0])}n{max(c[0])}-T{c[1]}H{c[2]}G{c[3]}d{c[4]}bs{c[5]}")
def test_attention(case, kind):
    lens, T, H, G, d, bs = case
    S = len(lens)
    cache, table, rows = make_cache(S, H, d, bs, lens, kind, 11 + d)
    q = rnd((S, T, H * G, d), FP if kind == "fp32" else BF, 3, scale=1.5)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = pkg.alloc_attention_workspace(q, H, table.shape[1] * bs)
    out, lse = attend(kind, q, cache, table, lens_d, lse=True, workspace=ws)
    assert status(ws) == 0
    check_attention(kind, q, out, lse, rows, lens, 1 / math.sqrt(d), cache)
    # a tight bound on the rows cuts the work otherwise; another scale; strided q and out
    tight = max(max(lens), 1)
    fused = torch.zeros(S, T, 3, H * G, d, dtype=q.dtype, device=DEV)
    fused[:, :, 1] = q
    buf = torch.full((S, T, 2, H * G, d), 4.0, dtype=q.dtype, device=DEV)
    ws2 = pkg.alloc_attention_workspace(q, H, tight)
    out2, lse2 = attend(kind, fused[:, :, 1], cache, table, lens_d, max_rows=tight, scale=0.3,
                        out=buf[:, :, 1], lse=True, workspace=ws2)
    assert status(ws2) == 0 and (buf[:, :, 0] == 4.0).all()
    check_attention(kind, q, out2, lse2, rows, lens, 0.3, cache)


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 3.0])
def test_attention_scales(kind, scale):
    """Negative scales turn the order of the logits, zero makes a mean."""
    lens, T, H, G, d, bs = [300, 77], 2, 2, 3, 64, 16
    cache, table, rows = make_cache(2, H, d, bs, lens, kind, 15)
    q = rnd((2, T, H * G, d), FP if kind == "fp32" else BF, 3, scale=2.0)
    out, lse = attend(kind, q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale, lse=True)
    check_attention(kind, q, out, lse, rows, lens, scale, cache)


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
def test_attention_keeps_hidden_rows_out(kind):
    """A NaN or an infinity in a row that only the later of the new tokens see
    does not reach the earlier ones."""
    lens, T, H, G, d, bs = [37, 5], 4, 1, 4, 64, 16
    cache, table, rows = make_cache(2, H, d, bs, lens, kind, 5)
    q = rnd((2, T, G, d), FP if kind == "fp32" else BF, 3)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = attend(kind, q, cache, table, lens_d)
    for s in range(2):  # the newest row: seen by the last token alone
        blk, r = int(table[s, (lens[s] - 1) // bs]), (lens[s] - 1) % bs
        if kind == "q4":
            cache.V_scales[blk, :, r] = float("nan")
        else:
            cache[1][blk, :, r, ::2] = float("nan")
            cache[1][blk, :, r, 1::2] = float("inf")
    out = attend(kind, q, cache, table, lens_d)
    assert torch.equal(out[:, :-1], clean[:, :-1])
    assert not torch.isfinite(out[:, -1]).any()


@pytest.mark.parametrize("kind", ["bf16", "q4", "fp32"])
def test_attention_extreme_logits(kind):
    """Large logits of both signs, growing along the row (the running maximum
    moves often), and keys that leave one row only."""
    H, d, bs, n = 1, 64, 16, 700
    cache, table, rows = make_cache(1, H, d, bs, [n], kind, 6)
    q = rnd((1, 1, 2, d), FP if kind == "fp32" else BF, 3, scale=40.0)
    lens_d = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = attend(kind, q, cache, table, lens_d, lse=True)
    check_attention(kind, q, out, lse, rows, [n], 1 / 8, cache)
    if kind != "q4":
        # masked by the caller's own keys: logits of -inf count nothing
        K, V = cache
        K2 = K.clone()
        K2[..., 0] = torch.where(torch.arange(K.shape[0] * bs, device=DEV).view(-1, 1, bs) % 3 == 0,
                                 torch.finfo(K.dtype).min, 0.0).to(K.dtype)
        q2 = q.clone()
        q2[..., 0] = 1e3  # 1e3 * lowest: -inf in fp32
        ids = table[0, :-(-n // bs)].long().cpu()
        krows = [K2.double().cpu()[ids].transpose(0, 1).reshape(H, -1, d)[:, :n]]
        out, lse = attend(kind, q2, (K2, V), table, lens_d, lse=True)
        z = (q2[0, 0].double().cpu().view(1, 2, d) @ krows[0].mT) / 8
        assert (z.abs().amax() > 3.4e38)
        z[z.abs() > 3.4e38] = -math.inf
        p = torch.softmax(z, -1)
        e = (p @ rows[1][0]).view(1, 1, 2, d)
        A = (p @ rows[1][0].abs()).view(1, 1, 2, d)
        L = (q2[..., 1:].double().cpu().abs().view(1, 2, d - 1) @ krows[0][..., 1:].abs().mT).amax()
        delta = float(L) * (d + 4) * ref.U32 / 8 + 64 * ref.U32
        tol = 2 * delta * A + 2 * (ref.U16 if kind == "bf16" else 2.0 ** -16) * (A + e.abs())
        assert ((out.double().cpu() - e).abs() <= tol).all()


def test_q4_attention_of_any_magnitude():
    """V's scales far from 1 (a power of two on all of V turns up in the output)
    and growing along the row (rows 2^60 smaller than others count as they
    should)."""
    lens, H, G, d, bs = [500, 37], 1, 3, 128, 16
    cache, table, rows = make_cache(2, H, d, bs, lens, "q4", 25, junk=False)
    q = rnd((2, 1, H * G, d), BF, 3)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    keep = cache.V_scales.clone()
    for k in (-60, -20, 33, 90):
        # (not bit for bit: the reference of the sums moves with the scales, and so do the
        # roundings of its exponentials)
        cache.V_scales.copy_(keep * 2.0 ** k)
        out, lse = attend("q4", q, cache, table, lens_d, lse=True)
        check_attention("q4", q, out, lse, [rows[0], [x * 2.0 ** k for x in rows[1]]], lens, 1 / math.sqrt(d), cache)
    # the first rows tiny, the last large: the running bound moves, and the tiny ones still
    # give their part of the sum of probabilities
    grow = torch.ones(keep.shape[0], bs, dtype=torch.float64)
    for s in range(2):
        for r in range(lens[s]):
            grow[int(table[s, r // bs]), r % bs] = 2.0 ** (r % 7 * 10 - 60 + (60 if r > lens[s] // 2 else 0))
    cache.V_scales.copy_((keep.double().cpu() * grow[:, None, :, None, None]).to(BF).to(DEV))
    vv = ref.values(cache.V_codes, cache.V_scales)
    nb = -(-max(lens) // bs)
    rows[1] = [vv[table[s, :nb].long().cpu().clamp(0, vv.shape[0] - 1)].transpose(0, 1).reshape(H, nb * bs, d)[:, :lens[s]]
               for s in range(2)]
    out, lse = attend("q4", q, cache, table, lens_d, lse=True)
    check_attention("q4", q, out, lse, rows, lens, 1 / math.sqrt(d), cache)


def test_q4_attention_of_any_query():
    """Queries far from 1 against keys as far the other way (the logits are the
    same), rows of one call of different magnitudes, elements of a row 2^20
    apart, and rows of zeros."""
    lens, H, G, d, bs = [500, 37], 1, 3, 128, 16
    cache, table, rows = make_cache(2, H, d, bs, lens, "q4", 26, junk=False)
    q = rnd((2, 1, H * G, d), BF, 3)
    q[..., 1::3] *= 2.0 ** -20
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    keep = cache.K_scales.clone()
    for k in (-100, -40, 60, 100):
        cache.K_scales.copy_(keep * 2.0 ** -k)
        out, lse = attend("q4", q * 2.0 ** k, cache, table, lens_d, lse=True)
        check_attention("q4", q * 2.0 ** k, out, lse, [[x * 2.0 ** -k for x in rows[0]], rows[1]], lens, 1 / math.sqrt(d), cache)
    cache.K_scales.copy_(keep)
    mixed = q.clone()
    mixed[:, :, 0] = 0
    mixed[0, :, 1] *= 2.0 ** -110
    mixed[1, :, 2] *= 4
    out, lse = attend("q4", mixed, cache, table, lens_d, lse=True)
    check_attention("q4", mixed, out, lse, rows, lens, 1 / math.sqrt(d), cache)
    # a row of the largest numbers sees the key nearest to it alone, the others theirs
    mixed[0, 0, 1] = q[0, 0, 1] * 2.0 ** 124
    out, lse = attend("q4", mixed, cache, table, lens_d, lse=True)
    best = (rows[0][0][0] @ mixed[0, 0, 1].double().cpu()).argmax()
    e = rows[1][0][0][best]
    # (p = 1: the output's rounding, and fp32 sums of scale * code, low and 8 * scale)
    assert ((out[0, 0, 1].double().cpu() - e).abs() <= 2.0 ** -8 * e.abs() + 2.0 ** -20 * e.abs().amax()).all()
    small = mixed.clone()
    small[0, 0, 1] = 0
    o2, l2 = attend("q4", small, cache, table, lens_d, lse=True)
    check_attention("q4", small, o2, l2, rows, lens, 1 / math.sqrt(d), cache)
    out[0, 0, 1] = o2[0, 0, 1]
    # (each within 2^-8 of the values' magnitude and of the output, and less for the rest)
    assert ((out - o2).abs() <= 2.0 ** -5 * max(float(x.abs().max()) for x in rows[1])).all()


def test_attention_bad_blocks_and_lens():
    """Ids that name no block: recorded, their rows skipped.  lens past
    max_rows is recorded and cut, a negative one counts as none."""
    lens, H, G, d, bs = [100, 60, 30], 2, 2, 64, 16
    for kind in ("bf16", "q4", "fp32"):
        cache, table, rows = make_cache(3, H, d, bs, lens, kind, 8)
        q = rnd((3, 1, H * G, d), FP if kind == "fp32" else BF, 4)
        ws = pkg.alloc_attention_workspace(q, H, 100)
        table[0, 2] = 1 << 20
        lens_d = torch.tensor([100, -1, 30], dtype=torch.int32, device=DEV)
        out, lse = attend(kind, q, cache, table, lens_d, max_rows=100, lse=True, workspace=ws)
        assert status(ws) == rkv.RKV_ERR_DEVICE and status(ws) == 0
        cut = [[torch.cat([x[0][:, :32], x[0][:, 48:]], 1), x[1][:, :0], x[2]] for x in rows]
        check_attention(kind, q, out, lse, cut, [84, 0, 30], 1 / 8, cache)
        lens_d = torch.tensor([50, 60, 30], dtype=torch.int32, device=DEV)
        out, lse = attend(kind, q[2:], cache, table[2:], lens_d[:1], max_rows=30, lse=True, workspace=ws)
        assert status(ws) == rkv.RKV_ERR_DEVICE
        check_attention(kind, q[2:], out, lse, [[r[2]] for r in rows], [30], 1 / 8, cache)


def test_long_offsets():
    """Pools whose bytes and elements pass 32 bits: the last blocks of a pool
    of 2.7e9 elements, paged and at 4 bits."""
    H, d, bs = 8, 128, 128
    blocks = 20600  # x 131072 elements
    lens, nb = [300], 3
    table = torch.tensor([[blocks - 1, blocks - 3, blocks - 2]], dtype=torch.int32, device=DEV)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = rnd((1, 300, H, d), BF, 1), rnd((1, 300, H, d), BF, 2)
    q = rnd((1, 1, H, d), BF, 3)
    ws = pkg.alloc_attention_workspace(q, H, 300)
    K = torch.empty(blocks, H, bs, d, dtype=BF, device=DEV)
    V = torch.empty_like(K)
    pkg.rkv_paged_append(K, V, k, v, table, lens_d, workspace=ws)
    out, lse = pkg.rkv_paged_attention(q, K, V, table, lens_d, max_rows=300, lse=True, workspace=ws)
    assert status(ws) == 0
    rows = [[x[0].double().cpu().transpose(0, 1)] for x in (k, v)]
    check_attention("bf16", q, out, lse, rows, lens, 1 / math.sqrt(d))
    del K, V
    blocks4 = 4 * blocks  # 64 bytes a row: 5.4e9 bytes of codes a side
    c = pkg.alloc_q4_cache(blocks4, H, bs, d)
    table4 = table - blocks + blocks4
    pkg.rkv_q4_append(c, k, v, table4, lens_d, workspace=ws)
    kk, vv = pkg.rkv_q4_read(c, table4, lens_d, 300, dtype=FP)
    for x, y in ((k, kk), (v, vv)):
        e = x[0].double().cpu().transpose(0, 1)
        code, s, lo = ref.quantise(e)
        assert ((y.double().cpu() - e).abs() <= s.repeat_interleave(32, -1) * 0.51).all()
    out, lse = pkg.rkv_q4_attention(q, c, table4, lens_d, max_rows=300, lse=True, workspace=ws)
    assert status(ws) == 0
    small = pkg.Q4Cache(*[t[blocks4 - 3:].contiguous() for t in (c.K_codes, c.K_scales, c.V_codes, c.V_scales)])
    check_attention("q4", q, out, lse, [[kk.double().cpu()], [vv.double().cpu()]], lens,
                    1 / math.sqrt(d), small)


# ---------------------------------------------------------------- together --

def test_decode_loop_with_compression():
    """Prompt, steps, compression, steps: a paged bf16 cache written by the
    append, read by the attention and pruned by rkv_paged_compress stays equal
    to a plain list of rows; rows and positions part after the compression."""
    S, H, G, d, bs = 2, 2, 4, 128, 16
    n, budget, steps = 150, 100, 3
    plan, f = pkg.RopePlan(d), ref.freqs(d)
    mb = 12
    table = torch.randperm(S * mb, generator=gen(1)).view(S, mb).to(torch.int32).to(DEV)
    K = torch.zeros(S * mb, H, bs, d, dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    k, v = rnd((S, n, H, d), BF, 2), rnd((S, n, H, d), BF, 3)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    pkg.rkv_paged_append(K, V, k, v, table, lens, rope=plan, workspace=ws)
    rows_k = ref.rotate(k.reshape(-1, H, d), torch.arange(n).repeat(S), f).to(BF).view(S, n, H, d)
    lists = [[rows_k[s].transpose(0, 1).double() for s in range(S)],
             [v[s].cpu().transpose(0, 1).double() for s in range(S)]]
    pos = n
    for phase in range(2):
        for i in range(steps):
            kn, vn, qn = (rnd((S, 1, h, d), BF, 10 * phase + i + j) for j, h in ((20, H), (40, H), (60, H * G)))
            lens += 1
            p = torch.full((S,), pos, dtype=torch.int32, device=DEV)
            qr = pkg.rkv_paged_append(K, V, kn, vn, table, lens, rope=plan, positions=p, q=qn, workspace=ws)
            out, lse = pkg.rkv_paged_attention(qr, K, V, table, lens, max_rows=mb * bs, lse=True, workspace=ws)
            assert status(ws) == 0
            kr = ref.rotate(kn.view(S, H, d), p, f).to(BF).double()
            for s in range(S):
                lists[0][s] = torch.cat([lists[0][s], kr[s][:, None]], 1)
                lists[1][s] = torch.cat([lists[1][s], vn[s].double().cpu().view(H, 1, d)], 1)
            ln = lens.tolist()
            # the kernel's own rows differ from the plain ones by a rounding of K at most
            mine = [[x[table[s].long()].transpose(0, 1).reshape(H, -1, d)[:, :ln[s]].double().cpu()
                     for s in range(S)] for x in (K, V)]
            for s in range(S):
                assert ((mine[0][s] - lists[0][s]).abs() <= 2.0 ** -7 * lists[0][s].abs() + 1e-5).all()
                assert torch.equal(mine[1][s], lists[1][s])
            check_attention("bf16", qr, out, lse, mine, ln, 1 / math.sqrt(d))
            pos += 1
        if phase == 0:
            q_obs = rnd((S * H, G, 8, d), BF, 99)
            idx, freed = pkg.rkv.rkv_paged_compress(K, V, q_obs, table, int(lens[0]), budget)
            assert freed.shape[1] == -(-int(lens[0]) // bs) - -(-budget // bs)
            # the freed blocks come back at the table's end as a serving loop would reuse them
            for s in range(S):
                keep = -(-budget // bs)
                table[s, keep:keep + freed.shape[1]] = freed[s]
            lists = [[torch.stack([x[s][h][idx[s * H + h].long().cpu()] for h in range(H)])
                      for s in range(S)] for x in mine]
            lens.fill_(budget)


def test_compress_into_four_bits():
    """A prompt compressed by rkv_compress, its kept rows held at 4 bits,
    further tokens appended and attended over; and the 4-bit rows read back
    are scored by rkv_score as any keys."""
    S, H, G, d, n, budget = 2, 2, 4, 64, 200, 128
    K, V = rnd((S * H, n, d), BF, 1), rnd((S * H, n, d), BF, 2)
    Qo = rnd((S * H, G, 8, d), BF, 3)
    oK, oV, _ = pkg.rkv_compress(K, V, Qo, n, budget)
    kept = [x.view(S, H, n, d)[:, :, :budget].transpose(1, 2) for x in (oK, oV)]
    mb = 10
    c = pkg.alloc_q4_cache(S * mb, H, 16, d)
    table = torch.arange(S * mb, dtype=torch.int32, device=DEV).view(S, mb)
    lens = torch.full((S,), budget, dtype=torch.int32, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    pkg.rkv_q4_append(c, kept[0], kept[1], table, lens, workspace=ws)
    plan = pkg.RopePlan(d)
    for i in range(3):
        kn, vn, qn = rnd((S, 1, H, d), BF, 30 + i), rnd((S, 1, H, d), BF, 40 + i), rnd((S, 1, H * G, d), BF, 50 + i)
        lens += 1
        p = torch.full((S,), n + i, dtype=torch.int32, device=DEV)
        qr = pkg.rkv_q4_append(c, kn, vn, table, lens, rope=plan, positions=p, q=qn, workspace=ws)
        out, lse = pkg.rkv_q4_attention(qr, c, table, lens, lse=True, workspace=ws)
        assert status(ws) == 0
        m = budget + i + 1
        rk, rv = pkg.rkv_q4_read(c, table, lens, m, dtype=FP, workspace=ws)
        rows = [[x.view(S, H, m, d)[s].double().cpu() for s in range(S)] for x in (rk, rv)]
        check_attention("q4", qr, out, lse, rows, [m] * S, 1 / 8, c)
    back, _ = pkg.rkv_q4_read(c, table, lens, budget)
    I, R, Z = pkg.rkv_score(back, Qo, budget)
    assert torch.isfinite(I).all() and torch.isinf(Z[:, -8:]).all()


@pytest.mark.parametrize("S", [3, 45])  # in one launch, and with pieces that a second one joins
def test_streams_graphs_and_two_calls_at_once(S):
    """Calls on a stream of their own, captured and replayed on new values,
    and two calls at once with a workspace each."""
    H, G, d, bs, n = 2, 4, 128, 16, 400
    cache, table, rows = make_cache(S, H, d, bs, [n] * S, "bf16", 3, junk=False)
    K, V = cache
    plan = pkg.RopePlan(d)
    k, v = rnd((S, 1, H, d), BF, 5), rnd((S, 1, H, d), BF, 6)
    q = rnd((S, 1, H * G, d), BF, 7)
    oq, out = torch.empty_like(q), torch.empty_like(q)
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    pos = torch.full((S,), 77, dtype=torch.int32, device=DEV)
    ws = pkg.alloc_attention_workspace(q, H, 400)

    def step(o, w, stream=None):
        pkg.rkv_paged_append(K, V, k, v, table, lens, rope=plan, positions=pos, q=q, out_q=oq,
                             workspace=w, stream=stream)
        pkg.rkv_paged_attention(oq, K, V, table, lens, max_rows=n, out=o, workspace=w, stream=stream)
    step(out, ws)
    torch.cuda.synchronize()
    want = out.clone()
    st = torch.cuda.Stream()
    out.zero_()
    st.wait_stream(torch.cuda.current_stream())
    step(out, ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, ws)
    for seed in (8, 9):
        q.copy_(rnd(q.shape, BF, seed))
        pos.fill_(1000 + seed)
        lens.fill_(n - seed)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(out, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    # two calls at once
    q2 = rnd(q.shape, BF, 10)
    one, two = torch.empty_like(q), torch.empty_like(q)
    w2 = pkg.alloc_attention_workspace(q, H, n)
    a = pkg.rkv_paged_attention(q, K, V, table, lens, max_rows=n, workspace=ws).clone()
    b = pkg.rkv_paged_attention(q2, K, V, table, lens, max_rows=n, workspace=ws).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        pkg.rkv_paged_attention(q, K, V, table, lens, max_rows=n, out=one, workspace=ws, stream=s1)
        pkg.rkv_paged_attention(q2, K, V, table, lens, max_rows=n, out=two, workspace=w2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(one, a) and torch.equal(two, b) and status(ws) == 0 and status(w2) == 0


@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("S", [3, 45])
def test_calls_that_depend_on_the_one_before(S, kind):
    """Each call's queries are the last one's output, its lengths and its cache
    just written: on a stream and captured (behind a memset, and where two
    streams meet) the bits of calls waited for one by one."""
    H, G, d, bs, n = 2, 4, 128, 16, 400
    cache, table, rows = make_cache(S, H, d, bs, [n] * S, kind, 3, junk=False)
    q = rnd((S, 1, H * G, d), BF, 7)
    x = [torch.empty_like(q) for _ in range(6)]
    k, v = rnd((S, 1, H, d), BF, 5), rnd((S, 1, H, d), BF, 6)
    lens = torch.empty(S, dtype=torch.int32, device=DEV)
    ws = pkg.alloc_attention_workspace(q, H, n)
    append = pkg.rkv_q4_append if kind == "q4" else pkg.rkv_paged_append
    side = torch.cuda.Stream()

    def run(wait):
        for i, out in enumerate(x):
            lens.zero_()
            lens.add_(n - 60 * i)
            if i % 2:
                append(*((cache,) if kind == "q4" else cache), k, v, table, lens, workspace=ws)
            wait()
            if i == 4:  # two streams meet before the call
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    lens.sub_(7)
                torch.cuda.current_stream().wait_stream(side)
            out.fill_(3.0)
            attend(kind, q if i == 0 else x[i - 1], cache, table, lens, max_rows=n, out=out, workspace=ws)
            wait()
    run(torch.cuda.synchronize)  # (its appends change rows that its first call read)
    run(torch.cuda.synchronize)
    want = [t.clone() for t in x]
    run(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(x, want)) and status(ws) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for _ in range(3):
        for t in x:
            t.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(x, want)) and status(ws) == 0
    # the memset right before the call
    g2 = torch.cuda.CUDAGraph()
    lens.fill_(n)
    torch.cuda.synchronize()
    a = attend(kind, q, cache, table, lens, max_rows=n, workspace=ws).clone()
    out = torch.empty_like(a)
    with torch.cuda.graph(g2):
        out.zero_()
        attend(kind, q, cache, table, lens, max_rows=n, out=out, workspace=ws)
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)


def test_token_calls_that_depend_on_the_one_before():
    """Rotations of a rotation's output, written to a 4-bit cache and read back
    as the next one's input, over tokens that fill the device several times: the
    bits of calls waited for one by one, on a stream and captured."""
    S, n, H, d, bs = 4, 2048, 4, 128, 64
    plan = pkg.RopePlan(d)
    pos = torch.arange(S * n, dtype=torch.int32, device=DEV)
    table = torch.arange(S * n // bs, dtype=torch.int32, device=DEV).view(S, -1)
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    c = pkg.alloc_q4_cache(S * n // bs, H, bs, d)
    start = rnd((S * n, H, d), BF, 4)
    x = [torch.empty_like(start) for _ in range(2)]
    k, v = (torch.empty(S * H, n, d, dtype=BF, device=DEV) for _ in range(2))

    def run(wait):
        x[0].copy_(start)
        for i in range(3):
            pkg.rkv_rope_apply(plan, pos, x[0], out_q=x[1])
            wait()
            pkg.rkv_rope_apply(plan, pos, x[1], out_q=x[1], inverse=i == 1)
            wait()
            pkg.rkv_q4_append(c, x[1].view(S, n, H, d), x[0].view(S, n, H, d), table, lens)
            wait()
            pkg.rkv_q4_read(c, table, lens, n, out_K=k, out_V=v)
            wait()
            rows = lambda t: t.view(S, H, n, d).transpose(1, 2)  # noqa: E731
            pkg.rkv_rope_apply(plan, pos, rows(k), rows(v), out_q=x[0].view(S, n, H, d), out_k=x[1].view(S, n, H, d))
            wait()
    run(torch.cuda.synchronize)
    want = [t.clone() for t in (*x, k, v)]
    for _ in range(3):
        run(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*x, k, v), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for t in (*x, k, v):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*x, k, v), want))


def test_same_result_every_time():
    for kind in ("bf16", "q4", "fp32"):
        lens = [3000, 17]
        cache, table, rows = make_cache(2, 1, 64, 16, lens, kind, 4)
        q = rnd((2, 2, 4, 64), FP if kind == "fp32" else BF, 3)
        lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
        a = attend(kind, q, cache, table, lens_d).clone()
        for _ in range(5):
            assert torch.equal(attend(kind, q, cache, table, lens_d), a)


def test_timing_names_the_kernels():
    rkv.rkv_timing_enable(True)
    try:
        rkv.rkv_timing_read()
        cache, table, rows = make_cache(1, 1, 64, 16, [40], "bf16", 4)
        q = rnd((1, 1, 2, 64), BF, 3)
        pkg.rkv_paged_attention(q, cache[0], cache[1], table, torch.tensor([40], dtype=torch.int32, device=DEV))
        pkg.rkv_rope_apply(pkg.RopePlan(64), torch.zeros(1, dtype=torch.int32, device=DEV), q[0])
        got = rkv.rkv_timing_read()
    finally:
        rkv.rkv_timing_enable(False)
    assert got["attention"][1] == 1 and got["rope"][1] == 1 and got["paged_append"][1] == 0
