"""Attention over shared prefixes and over 8-bit caches with logits of any size that
fp32 holds, as tests/test_gpu_attention_magnitudes.py has it for the other caches:
parts of the rows whose maxima differ, sums that pass from ordinary to far logits, and
ordinary keys under large queries."""

import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv
from tests import cache_ref as ref
from tests import prefix_ref, q8_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
SIZES = (0, 8, 13, 14, 15, 16, 18, 22, 25, 33, 60, 110)
FACTORS = (1.0, -0.75, 1.25, None)  # of a large head; None: 2^-k, an ordinary one beside them


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rnd(shape, dtype, seed):
    return torch.randn(*shape, generator=gen(seed)).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def factors(heads, k):
    return torch.tensor([FACTORS[i % 4] or 2.0 ** -k for i in range(heads)], dtype=torch.float64) * 2.0 ** k


def compare(z, v, out, lse, exact):
    """z [heads, rows] exact logits, v [rows, d]; exact: probabilities and output in fp32.

    A logit (to base 2) is off by 8 * 2^-24 of itself, which moves the weights unless the largest
    alone (with its equals) has any; the probabilities' rounding and the output's 2^-8 each.  An
    exponential of less than 2^-126 is 0, and what it is relative to lies up to 2^8 below the largest:
    n rows lose n 2^-118 of the largest value at most (where that row's own value is 0, no more is
    left of the sum)."""
    n = z.shape[1]
    le, P = torch.logsumexp(z, -1), torch.softmax(z, -1)
    e, A = P @ v, P @ v.abs()
    top = z.amax(-1, keepdim=True)
    same = (z == top).sum(-1)
    alone = (torch.exp((z - top).clamp(min=-700)).sum(-1) - same) < 1e-9
    off = torch.clamp(z.abs().amax(-1) * 8 * ref.U32, max=1.0)
    delta = torch.where(alone, torch.zeros_like(off), off) + 40 * ref.U32
    b = (2 * delta[:, None] + (n / 2 + 128) * ref.U32) * A
    b = b + n * 2.0 ** -118 * v.abs().amax()
    if not exact:
        b = b + ref.U16 * A
    b = b + (ref.U32 if exact else ref.U16) * (e.abs() + b)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - e).abs() <= b).all(), float(((got - e).abs() / b).max())
    assert ((lse.double().cpu() - le).abs() <= 16 * ref.U32 * (1 + le.abs()) + n * ref.U32).all()


def one_row_has_it(q, k, v, scale, out, lse):
    """q [heads, d], k and v [rows, d] in 64 bits: where a row is ahead of the others by more than the
    logits may be off (d products and the steps behind them, 2^-24 of sum |q| |k| each), the output is
    its value, rounded twice; the sum's log is off by as much as a logit."""
    z = q @ k.T * scale
    two, at = z.topk(2, -1)
    off = (q.abs() @ k.abs().T).amax(-1) * abs(scale) * (q.shape[-1] + 40) * ref.U32
    got = out.double().cpu()
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    found = 0
    for h in range(len(q)):
        if two[h, 0] - two[h, 1] > 2 * off[h] + 40:  # the others below e^-40
            found += 1
            e = v[at[h, 0]]
            assert ((got[h] - e).abs() <= 2.0 ** -7 * e.abs() + 2.0 ** -30 * v.abs().amax()).all()
    assert ((lse.double().cpu() - torch.logsumexp(z, -1)).abs() <= off + 1e-4 + 2.0 ** -20 * z.abs().amax(-1)).all()
    return found


# ---------------------------------------------------------------- prefixes --

PREFIX = [
    # prefix lens, groups, T, G, d, block, type
    ([700, 1300], [0, 20, 60], 1, 4, 128, 16, BF),   # tiles of 256 queries
    ([700, 1300], [0, 5, 11], 1, 4, 128, 64, BF),    # 128 or fewer: two shares of the rows
    ([9000], [0, 6], 3, 4, 64, 128, BF),
    ([4000], [0, 30], 2, 8, 64, 8, BF),
    ([700, 1300], [0, 5, 11], 1, 4, 128, 4, BF),     # CUDA cores
    ([500, 70], [0, 8, 12], 2, 4, 64, 16, FP),
]


class Prefixes:
    def __init__(self, plens, groups, T, G, d, bs, dt):
        self.plens, self.groups, self.T, self.G, self.d, self.dt = plens, groups, T, G, d, dt
        S = groups[-1] + 1  # the last without a prefix
        self.lens = [(7 * s) % 90 for s in range(S)]
        self.lens[-1] = 40
        pb, ob = -(-max(plens) // bs), -(-90 // bs)
        perm = torch.randperm(len(plens) * pb + S * ob, generator=gen(3)).to(torch.int32)
        self.ptable, self.table = perm[:len(plens) * pb].view(-1, pb), perm[len(plens) * pb:].view(S, ob)
        self.K, self.V = (rnd((perm.numel(), 1, bs, d), dt, 4 + i) for i in range(2))

    def call(self, q):
        ws = pkg.alloc_prefix_attention_workspace(q, 1, 128, len(self.plens), 16384)
        out = pkg.rkv_prefix_attention(q, self.K.to(DEV), self.V.to(DEV), self.ptable.to(DEV), ints(self.plens),
                                       self.table.to(DEV), ints(self.lens), cu_seqs=ints(self.groups), lse=True,
                                       workspace=ws, scale=0.3, max_rows=90)
        assert rkv.rkv_get_device_status(ws) == 0
        return out

    def seen(self, s, t):
        """K and V of token t of sequence s: its prefix, then its own rows."""
        p = prefix_ref.group_of(self.groups, s)
        own = [prefix_ref.rows_of(x, self.table[s:s + 1], self.lens[s:s + 1])[0][0] for x in (self.K, self.V)]
        own = [x[:max(0, self.lens[s] - self.T + t + 1)] for x in own]
        if p is None:
            return own
        pre = [prefix_ref.rows_of(x, self.ptable[p:p + 1], self.plens[p:p + 1])[0][0] for x in (self.K, self.V)]
        return [torch.cat(x) for x in zip(pre, own)]

    def tokens(self):
        S = len(self.lens)
        return [(s, t) for s in (0, 1, S // 2, S - 2, S - 1) for t in {0, self.T - 1}]


@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: f"p{max(c[0])}S{c[1][-1] + 1}T{c[2]}G{c[3]}d{c[4]}b{c[5]}{'f' if c[6] is FP else ''}")
def test_prefix_logits_of_any_size(case, order):
    """Keys whose first element is a whole number and the others 0, so that logits are exact; rising ones pass
    every maximum on the way."""
    c = Prefixes(*case)
    nb, _, bs, _ = c.K.shape
    c.K.zero_()
    whole = torch.randint(-60, 61, (nb, bs), generator=gen(9)).to(c.dt)
    c.K[:, 0, :, 0] = whole
    if order != "mixed":
        for p, n in enumerate(c.plens):
            x = torch.linspace(-60, 60, n).round().to(c.dt)
            x = x if order == "rising" else x.flip(0)
            for r in range(n):
                c.K[int(c.ptable[p, r // bs]), 0, r % bs, 0] = x[r]
    S = len(c.lens)
    scale = float(torch.tensor(0.3, dtype=FP))
    rows = {x: c.seen(*x) for x in c.tokens()}
    for k in SIZES:
        q = torch.zeros(S, c.T, c.G, c.d, dtype=c.dt)
        f = factors(c.G, k)
        q[..., 0] = f.to(c.dt)
        out, lse = c.call(q.to(DEV))
        for (s, t), (kk, vv) in rows.items():
            compare(f[:, None] * kk[None, :, 0] * scale, vv, out[s, t], lse[s, t], c.dt == FP)


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: f"p{max(c[0])}S{c[1][-1] + 1}T{c[2]}G{c[3]}d{c[4]}b{c[5]}{'f' if c[6] is FP else ''}")
def test_prefix_any_keys_and_large_queries(case):
    c = Prefixes(*case)
    q0 = rnd((len(c.lens), c.T, c.G, c.d), c.dt, 11)
    scale = float(torch.tensor(0.3, dtype=FP))
    rows = {x: c.seen(*x) for x in c.tokens()}
    found = 0
    for k in (3, 8, 14, 15, 17, 20, 27, 33, 60):
        q = q0 * 2.0 ** k
        out, lse = c.call(q.to(DEV))
        for (s, t), (kk, vv) in rows.items():
            found += one_row_has_it(q[s, t].double(), kk, vv, scale, out[s, t], lse[s, t])
    assert found > 60


# ------------------------------------------------------------------ 8 bits --

EIGHT = [([37], 1, 2, 64, 16), ([300, 5], 1, 4, 128, 16), ([1152], 1, 16, 128, 16), ([400], 8, 4, 64, 16),
         ([700, 1], 3, 2, 128, 64), ([9001], 1, 3, 64, 16), ([4000, 64, 3000] * 3, 2, 4, 128, 16)]


def eight(lens, d, bs, seed):
    """Arrays of a cache of ordinary rows, and a table."""
    S, nb = len(lens), -(-max(lens) // bs)
    table = torch.randperm(S * nb + 2, generator=gen(seed))[:S * nb].view(S, nb).to(torch.int32)
    arrays = []
    for i in range(2):
        codes, scales = q8_ref.quantise(rnd((S * nb + 2, 1, bs, d), BF, seed + i).double())
        arrays += [codes, scales]
    return arrays, table


def eight_rows(arrays, table, lens):
    return [[x[0] for x in q8_ref.rows_of(*arrays[2 * i:2 * i + 2], table, lens)] for i in range(2)]


def eight_call(arrays, table, lens, q, scale):
    cache = pkg.Q8Cache(*[x.to(DEV) for x in arrays])
    ws = pkg.alloc_attention_workspace(q, 1, max(lens))
    out = pkg.rkv_q8_attention(q, cache, table.to(DEV), ints(lens), max_rows=max(lens), scale=scale, lse=True, workspace=ws)
    assert rkv.rkv_get_device_status(ws) == 0
    return out


@pytest.mark.parametrize("case", EIGHT, ids=lambda c: f"S{len(c[0])}n{max(c[0])}T{c[1]}G{c[2]}d{c[3]}")
def test_eight_bit_logits_of_any_size(case):
    lens, T, G, d, bs = case
    arrays, table = eight(lens, d, bs, 21)
    codes, scales = arrays[0], arrays[1]
    codes.zero_()
    codes[..., 0] = torch.randint(-127, 128, codes.shape[:-1], generator=gen(5))
    scales.fill_(0.5)
    K, V = eight_rows(arrays, table, lens)
    scale = float(torch.tensor(0.3, dtype=FP))
    for k in SIZES:
        q = torch.zeros(len(lens), T, G, d, dtype=BF)
        f = factors(G, k)
        q[..., 0] = f.to(BF)
        out, lse = eight_call(arrays, table, lens, q.to(DEV), 0.3)
        for s, n in enumerate(lens):
            for t in range(T):
                see = n - T + t + 1
                if see <= 0:
                    assert (out[s, t] == 0).all()
                    continue
                compare(f[:, None] * K[s][None, :see, 0] * scale, V[s][:see], out[s, t], lse[s, t], False)


@pytest.mark.parametrize("lens", [[1345], [357] * 20, [9001, 60]], ids=lambda n: f"S{len(n)}n{max(n)}")
def test_eight_bit_any_keys_and_large_queries(lens):
    T, G, d, bs = 3, 2, 128, 16
    arrays, table = eight(lens, d, bs, 31)
    K, V = eight_rows(arrays, table, lens)
    q0 = rnd((len(lens), T, G, d), BF, 7)
    found = 0
    for k in (3, 8, 14, 17, 20, 27, 33, 60):
        q = q0 * 2.0 ** k
        out, lse = eight_call(arrays, table, lens, q.to(DEV), d ** -0.5)
        for s, n in enumerate(lens):
            for t in range(T):
                see = n - T + t + 1
                found += one_row_has_it(q[s, t].double(), K[s][:see], V[s][:see], d ** -0.5, out[s, t], lse[s, t])
    assert found > 20


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 100])
def test_eight_bit_values_of_any_size(G, size):
    """Values of 2^-100 and 2^100: the probabilities times the rows' scales keep their digits."""
    lens, T, d, bs = [1500, 33], 1 + (G == 16), 64, 16
    arrays, table = eight(lens, d, bs, 41)
    arrays[3] *= size
    K, V = eight_rows(arrays, table, lens)
    q = rnd((2, T, G, d), BF, 8)
    out, lse = eight_call(arrays, table, lens, q.to(DEV), d ** -0.5)
    e, el, A, L = ref.attention(q, [x[None] for x in K], [x[None] for x in V], lens, d ** -0.5)
    b, bl = ref.attention_bounds(e, el, A, L, d ** -0.5, d, max(lens), "bf16")
    assert ((out.double().cpu() - e).abs() <= b).all(), float(((out.double().cpu() - e).abs() / b).max())
    assert ((lse.double().cpu() - el).abs() <= bl).all()
