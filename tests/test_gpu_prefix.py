"""Attention over shared prefixes on the GPU against a plain 64-bit form: groups,
lengths, types, strides, hidden and broken rows; and a run with appends and the
compression."""
import math

import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from decode_kv_cache_02_gb300 import rkv
from tests import cache_ref as ref
from tests import prefix_ref

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


class Case:
    """Pools, tables and queries of a batch; groups as prefix_ref.group_of takes them."""

    def __init__(self, prefix_lens, groups, lens, T, H, G, d, bs, dt, seed=3):
        self.plens, self.groups, self.lens = prefix_lens, groups, lens
        self.T, self.H, self.G, self.d, self.bs, self.dt = T, H, G, d, bs, dt
        S, P = len(lens), len(prefix_lens)
        pb = max([1] + [-(-n // bs) for n in prefix_lens]) + 1
        ob = max([1] + [-(-n // bs) for n in lens])
        nb = P * pb + S * ob + 1
        perm = torch.randperm(nb, generator=gen(seed)).to(torch.int32)
        self.ptable = perm[: P * pb].view(P, pb)
        self.table = perm[P * pb: P * pb + S * ob].view(S, ob)
        self.K, self.V = rnd((nb, H, bs, d), dt, seed + 1), rnd((nb, H, bs, d), dt, seed + 2)
        self.K += rnd((H, 1, d), dt, seed + 5, 0.5)
        self.q = rnd((S, T, H * G, d), dt, seed + 4)

    def ws(self):
        return pkg.alloc_prefix_attention_workspace(self.q, self.H, self.table.shape[1] * self.bs, len(self.plens),
                                                    max(1, self.ptable.shape[1] * self.bs))

    def call(self, ws=None, cu=True, **kw):
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        kw.setdefault("q", self.q)
        kw.setdefault("lse", True)
        q = kw.pop("q")
        return pkg.rkv_prefix_attention(q, self.K, self.V, self.ptable.to(DEV), ints(self.plens), self.table.to(DEV),
                                        ints(self.lens), cu_seqs=ints(self.groups) if cu else None, workspace=ws, **kw)

    def compare(self, out, lse, scale=None, q=None, seqs=None):
        """seqs: of the first of the sequences alone."""
        scale = self.d ** -0.5 if scale is None else scale
        q = (self.q if q is None else q)[:seqs]
        pk, pv = (prefix_ref.rows_of(x, self.ptable, self.plens) for x in (self.K, self.V))
        ok, ov = (prefix_ref.rows_of(x, self.table, self.lens[:seqs]) for x in (self.K, self.V))
        e, el, A, L = prefix_ref.attention(q, pk, pv, self.groups, ok, ov, self.lens, scale)
        rows = max([0] + self.plens) + max(self.lens)
        b, bl = ref.attention_bounds(e, el, A, L, scale, self.d, max(rows, 1), "fp32" if self.dt == FP else "bf16")
        none = torch.isinf(el)
        assert torch.equal(torch.isinf(lse.cpu()), none)
        got = out.double().cpu()
        assert (got[none] == 0).all() and torch.isfinite(got).all()
        worst = ((got - e).abs() / b).max()
        assert worst <= 1, float(worst)
        assert ((lse.double().cpu() - el).abs()[~none] <= bl[~none]).all()


CASES = [
    # prefix lens, groups, own lens, T, H, G, d, block
    ([1], [0, 1], [1], 1, 1, 1, 128, 16),
    ([1], [0, 1], [0], 1, 1, 1, 64, 8),
    ([0], [0, 2], [0, 5], 1, 2, 2, 64, 8),                              # an empty prefix
    ([127, 128, 129], [0, 2, 3, 6], [5, 1, 0, 64, 65, 3], 1, 2, 4, 128, 16),
    ([300, 0, 17, 700], [0, 4, 5, 5, 9], [9, 8, 7, 6, 5, 4, 3, 2, 1, 40, 0], 1, 3, 5, 128, 32),  # empty group, two alone
    ([1000], [0, 0], [3, 900], 1, 2, 3, 64, 16),                        # a prefix nobody has
    ([640], [0, 40], list(range(40)), 1, 8, 4, 128, 128),               # 160 queries
    ([900, 333], [0, 50, 70], [7 + i % 13 for i in range(70)], 1, 2, 7, 128, 8),   # 350 and 140 queries
    ([513], [0, 9], [8, 3, 0, 1, 100, 70, 64, 65, 2], 8, 2, 4, 64, 16),  # new tokens, own rows fewer than them
    ([200, 77], [0, 1, 3], [64, 70, 1], 64, 1, 2, 64, 64),              # 64 new tokens
    ([257], [0, 6], [1] * 6, 5, 1, 16, 128, 256),                       # 480 queries, blocks past a tile
    ([5000], [0, 3], [30, 1, 2], 1, 1, 1, 128, 16),                     # few queries, many runs
    ([2500] * 5, [0, 1, 2, 3, 4, 5], [300, 20, 1, 0, 77], 2, 4, 2, 128, 1024),
    ([20000], [0, 33], [5] * 33, 1, 2, 4, 64, 128),
    ([400, 70, 9], [0, 90, 95, 96], [6 + i % 9 for i in range(97)], 1, 1, 8, 128, 16),  # teams with members without queries
    ([300, 900, 40, 700, 65, 129], [0, 4, 70, 73, 139, 200, 203], [i % 4 for i in range(204)], 1, 8, 4, 128, 64),  # one or two groups of queries in turn
    ([150, 600], [0, 9, 12], [64 + i for i in range(12)], 64, 1, 8, 64, 32),            # 4608 and 1536 queries
    ([1, 2, 3] * 30, list(range(0, 182, 2)) , [1 + i % 3 for i in range(180)], 1, 1, 1, 64, 8),  # many prefixes
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"p{len(c[0])}x{max(c[0])}-s{len(c[2])}-t{c[3]}-{c[4]}x{c[5]}x{c[6]}-b{c[7]}")
def test_prefix_attention(case, dt):
    c = Case(*case, dt)
    ws = c.ws()
    out, lse = c.call(ws)
    assert status(ws) == 0
    c.compare(out, lse)
    again, lse2 = c.call(ws)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert status(ws) == 0


@pytest.mark.parametrize("d, bs", [(128, 128), (128, 8), (64, 64), (64, 16)])
@pytest.mark.parametrize("queries", [70, 200])
def test_long_pieces(d, bs, queries):
    """A block's share of a prefix goes through its ring of tiles many times, call after call: the same bits, and
    those of the definition."""
    c = Case([60001, 9000], [0, queries - 5, queries], [3 + i % 5 for i in range(queries)], 1, 8, 1, d, bs, BF)
    ws = [c.ws() for _ in range(2)]
    first, lse = c.call(ws[0])
    c.compare(first[:3], lse[:3], seqs=3)
    again = [c.call(w)[0] for _ in range(20) for w in ws]
    assert all(torch.equal(x, first) for x in again) and status(ws[0]) == 0 and status(ws[1]) == 0


@pytest.mark.parametrize("bs", [1, 2, 4])
def test_small_blocks(bs):
    c = Case([70, 133], [0, 3, 5], [9, 0, 4, 2, 1], 2, 2, 4, 128, bs, BF)
    out, lse = c.call()
    c.compare(out, lse)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_without_cu_seqs(dt):
    c = Case([70, 300, 128], [0, 4, 8, 12], [5] * 12, 1, 2, 4, 128, 16, dt)
    a, la = c.call()
    b, lb = c.call(cu=False)
    assert torch.equal(a, b) and torch.equal(la, lb)
    c.compare(b, lb)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 6.0])
def test_scales_strides_and_bounds(scale, dt):
    """Signs of the scale; queries and outputs as slices; tighter bounds on the lengths."""
    c = Case([400, 90], [0, 30, 41], [3 + i for i in range(41)], 2, 2, 4, 128, 16, dt)
    S, T, hq, d = c.q.shape
    wide = rnd((S, T, hq, 2 * d), dt, 77)
    q = wide[..., d:]
    o = torch.zeros(S, hq, T, d, dtype=dt, device=DEV).transpose(1, 2)
    out, lse = c.call(q=q, scale=scale, out=o, max_rows=43, max_prefix_rows=400)
    assert out.data_ptr() == o.data_ptr()
    c.compare(out, lse, scale, q)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_large_logits(dt):
    """Logits up to 2^40: the weights of the rows at the largest one are those of their differences (keys with one
    element large, so that the products are exact)."""
    c = Case([300], [0, 40], [6] * 40, 1, 1, 4, 64, 16, dt)
    for big in (2.0 ** 20, 2.0 ** 40):
        c.K.zero_()
        c.K[..., 0] = big
        c.q.zero_()
        c.q[..., 0] = 1.0
        c.q[3, 0, 1, 0] = -1.0
        out, lse = c.call(scale=1.0)
        pv, ov = (prefix_ref.rows_of(c.V, t, n)[0] for t, n in ((c.ptable, c.plens), (c.table, c.lens)))
        own = prefix_ref.rows_of(c.V, c.table, c.lens)
        for s in (0, 3, 39):
            mean = torch.cat([pv, own[s]], 1).mean(1)
            size = torch.cat([pv, own[s]], 1).abs().mean(1)
            # all weights are equal: the probabilities' rounding and the output's, 2^-8 each (fp32: sums of 306)
            lim = (2 * ref.U16 if dt == BF else 400 * ref.U32) * size + 1e-30
            assert ((out[s, 0].double().cpu() - mean).abs() <= lim).all(), (big, s)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_what_hidden_rows_hold(dt):
    """Rows behind a prefix in its last block and behind the own rows, and blocks of nobody, may hold anything."""
    c = Case([203, 128, 9], [0, 20, 30, 33], [17] * 33, 1, 2, 8, 128, 32, dt)
    a, la = c.call()
    used = torch.zeros(c.K.shape[0], c.bs, dtype=torch.bool)
    for table, lens in ((c.ptable, c.plens), (c.table, c.lens)):
        for s, n in enumerate(lens):
            for r in range(n):
                used[int(table[s, r // c.bs]), r % c.bs] = True
    for bad in (math.nan, math.inf):
        for x in (c.K, c.V):
            x.transpose(1, 2)[~used.to(DEV)] = bad
        b, lb = c.call()
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_not_finite_stays_with_its_own(dt):
    """A NaN in one prefix, one sequence's rows or one query: that prefix's, sequence's or query's outputs alone;
    infinite logits to the left leave nothing."""
    c = Case([260, 200], [0, 20, 40], [9] * 40, 1, 2, 4, 64, 16, dt)
    clean, lc = c.call()
    at = lambda t, r, s: (int(t[s, r // c.bs]), r % c.bs)  # noqa: E731
    b, o = at(c.ptable, 131, 0)
    keep = c.V[b, 1, o, 5].clone()
    c.V[b, 1, o, 5] = math.nan
    out, _ = c.call()
    wrong = torch.zeros_like(out, dtype=torch.bool)
    wrong[:20, :, 4:, 5] = True
    assert torch.equal(torch.isnan(out), wrong) and torch.equal(out[~wrong], clean[~wrong])
    c.V[b, 1, o, 5] = keep
    b, o = at(c.table, 3, 25)
    keep = c.K[b, 0, o, 7].clone()
    c.K[b, 0, o, 7] = math.nan
    out, _ = c.call()
    wrong.zero_()
    wrong[25, :, :4] = True
    assert torch.equal(torch.isnan(out), wrong) and torch.equal(out[~wrong], clean[~wrong])
    c.K[b, 0, o, 7] = keep
    c.q[2, 0, 3, 0] = math.nan
    out, _ = c.call()
    wrong.zero_()
    wrong[2, 0, 3] = True
    assert torch.equal(torch.isnan(out), wrong) and torch.equal(out[~wrong], clean[~wrong])
    # every logit of a query -inf: nothing is seen
    c.q[2, 0, 3] = 1.0
    c.K.zero_()
    c.K[..., 0] = -math.inf
    c.q[..., 0] = 1.0
    c.q[..., 1:] = 0.0
    c.q[5, 0, 0, 0] = 0.5
    out, lse = c.call()
    assert (out == 0).all() and torch.isinf(lse).all() and (lse < 0).all()


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_bad_ids_lengths_and_groups(dt):
    c = Case([300, 50], [0, 30, 34], [20] * 34, 1, 2, 4, 128, 16, dt)
    ws = c.ws()
    good = c.ptable.clone()
    for bad in (-1, c.K.shape[0], 2 ** 31 - 1):
        c.ptable[0, 2] = bad
        out, lse = c.call(ws)
        assert status(ws) == 6 and status(ws) == 0
        # the block's rows are skipped
        keep = torch.ones(300, dtype=torch.bool)
        keep[32:48] = False
        pk, pv = ([x[0][:, keep], x[1]] for x in (prefix_ref.rows_of(y, good, c.plens) for y in (c.K, c.V)))
        ok, ov = (prefix_ref.rows_of(x, c.table, c.lens) for x in (c.K, c.V))
        e, el, A, L = prefix_ref.attention(c.q, pk, pv, c.groups, ok, ov, c.lens, c.d ** -0.5)
        b, _ = ref.attention_bounds(e, el, A, L, c.d ** -0.5, c.d, 320, "fp32" if dt == FP else "bf16")
        assert ((out.double().cpu() - e).abs() <= b).all()
    c.ptable.copy_(good)
    fine, _ = c.call(ws)
    assert status(ws) == 0
    # lengths past the bound or negative are cut
    bound = c.ptable.shape[1] * c.bs
    for n, same in ((bound + 1, bound), (-5, 0)):
        c.plens = [n, 50]
        a, la = c.call(ws)
        assert status(ws) == 6
        c.plens = [same, 50]
        b, lb = c.call(ws)
        assert status(ws) == 0 and torch.equal(a, b) and torch.equal(la, lb)
    c.plens = [300, 50]
    # groups that descend, begin behind 0 or end past the batch are cut, every sequence is in one
    for groups, same in (([0, 30, 99], [0, 30, 34]), ([0, 31, 5], [0, 31, 31]), ([3, 30, 34], [0, 30, 34]),
                         ([0, -7, 34], [0, 0, 34])):
        c.groups = groups
        a, la = c.call(ws)
        assert status(ws) == 6
        c.groups = same
        b, lb = c.call(ws)
        assert status(ws) == 0 and torch.equal(a, b) and torch.equal(la, lb)
    c.groups = [0, 30, 34]
    again, _ = c.call(ws)
    assert torch.equal(again, fine)


def test_same_as_without_a_prefix():
    """No prefixes, and prefixes of no rows: the rows of rkv_paged_attention, one rounding after the join."""
    c = Case([], [0], [300, 7, 0, 64], 1, 2, 4, 128, 16, BF)
    out, lse = c.call(cu=False)
    c.compare(out, lse)
    lt = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    plain, lp = pkg.rkv_paged_attention(c.q, c.K, c.V, c.table.to(DEV), lt, lse=True)
    assert torch.equal(out, plain) and torch.equal(lse, lp)
    assert pkg.rkv_prefix_attention(c.q[:0], c.K, c.V, c.ptable.to(DEV), lt[:0], c.table[:0].to(DEV), lt[:0]).shape == (0, 1, 8, 128)


def test_two_captured_graphs_and_streams():
    """Captured and replayed with a workspace each, and on two streams at once: the bits of the plain calls."""
    a = Case([700], [0, 40], [12] * 40, 1, 2, 4, 128, 16, BF, seed=1)
    b = Case([130, 90], [0, 9, 20], [40] * 20, 2, 2, 4, 64, 32, BF, seed=2)
    cs, plain, graphs, outs = (a, b), [], [], []
    for c in cs:
        plain.append(c.call(c.ws())[0])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for c in cs:
        ws, out = c.ws(), torch.zeros_like(c.q)
        args = (c.q, c.K, c.V, c.ptable.to(DEV), ints(c.plens), c.table.to(DEV), ints(c.lens))
        kw = dict(cu_seqs=ints(c.groups), out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.rkv_prefix_attention(*args, **kw)
        graphs.append((g, ws, args, kw))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, (g, *_x) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], plain[0]) and torch.equal(outs[1], plain[1])
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for s, (_g, _ws, args, kw) in zip(streams, graphs):
        pkg.rkv_prefix_attention(*args, stream=s, **kw)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], plain[0]) and torch.equal(outs[1], plain[1])


def test_run_with_appends_and_compression():
    """Samples of one prompt: the prompt appended once as a sequence of its own, the samples' tokens appended and
    attended step by step, their rows compressed in place (the prompt's blocks are no sequence's own), a step more."""
    N, H, G, d, bs, prompt, n, budget, n_obs = 3, 2, 4, 128, 16, 150, 160, 96, 8
    nb_p, nb_o = -(-prompt // bs), -(-(n + 4) // bs)
    perm = torch.randperm(nb_p + N * nb_o, generator=gen(9)).to(torch.int32).to(DEV)
    ptable, table = perm[:nb_p].view(1, nb_p).contiguous(), perm[nb_p:].view(N, nb_o).contiguous()
    K = torch.zeros(nb_p + N * nb_o, H, bs, d, dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    plan = pkg.RopePlan(d)
    plens = torch.tensor([prompt], dtype=torch.int32, device=DEV)
    pk, pv = rnd((1, prompt, H, d), BF, 1), rnd((1, prompt, H, d), BF, 2)
    pkg.rkv_paged_append(K, V, pk, pv, ptable, plens, rope=plan)
    lens = torch.full((N,), n, dtype=torch.int32, device=DEV)
    k, v = rnd((N, n, H, d), BF, 3), rnd((N, n, H, d), BF, 4)
    pos = (prompt + torch.arange(n, dtype=torch.int32, device=DEV)).repeat(N, 1)
    pkg.rkv_paged_append(K, V, k, v, table, lens, rope=plan, positions=pos)
    before = K[ptable[0].long()].clone()

    def step(at, lens, seed):
        nk, nv, q = rnd((N, 1, H, d), BF, seed), rnd((N, 1, H, d), BF, seed + 1), rnd((N, 1, H * G, d), BF, seed + 2)
        p = torch.full((N,), at, dtype=torch.int32, device=DEV)
        lens = lens + 1
        q = pkg.rkv_paged_append(K, V, nk, nv, table, lens, rope=plan, positions=p, q=q)
        out, lse = pkg.rkv_prefix_attention(q, K, V, ptable, plens, table, lens, lse=True)
        pks, pvs = (prefix_ref.rows_of(x, ptable.cpu(), [prompt]) for x in (K, V))
        oks, ovs = (prefix_ref.rows_of(x, table.cpu(), lens.tolist()) for x in (K, V))
        e, el, A, L = prefix_ref.attention(q, pks, pvs, [0, N], oks, ovs, lens.tolist(), d ** -0.5)
        b, bl = ref.attention_bounds(e, el, A, L, d ** -0.5, d, prompt + n + 2, "bf16")
        assert ((out.double().cpu() - e).abs() <= b).all() and ((lse.double().cpu() - el).abs() <= bl).all()
        return lens
    lens = step(prompt + n, lens, 20)
    Q = rnd((N * H, G, n_obs, d), BF, 5)
    idx, freed = rkv.rkv_paged_compress(K, V, Q, table, n + 1, budget, n_obs)[:2]
    assert (freed >= 0).all() and (table[:, -(-budget // bs):-(-(n + 1) // bs)] == -1).all()
    assert torch.equal(K[ptable[0].long()], before)
    table[:, budget // bs] = freed[:, 0]  # room for the next token, from what was handed back
    lens = torch.full((N,), budget, dtype=torch.int32, device=DEV)
    step(prompt + n + 1, lens, 30)


def test_python_refusals():
    c = Case([40, 50], [0, 2, 3], [3] * 3, 1, 1, 2, 64, 8, BF)
    with pytest.raises(ValueError):
        c.call(cu=False)                     # three sequences, two prefixes
    with pytest.raises(ValueError):
        c.call(q=c.q.float())
    with pytest.raises(ValueError):
        c.call(max_prefix_rows=0)
    with pytest.raises(ValueError):
        c.call(max_prefix_rows=(1 << 32) + 8)
    with pytest.raises(rkv.RkvError):
        c.call(max_prefix_rows=1000)         # past the table
    with pytest.raises(rkv.RkvError) as e:
        c.call(torch.zeros(512, dtype=torch.uint8, device=DEV))
    assert e.value.code == 3
    with pytest.raises(ValueError):
        pkg.rkv_prefix_attention_workspace_size(c.q, 1, 0, 1, 10)


def test_prefixes_that_share_blocks():
    """Two prefixes over the same blocks, at other lengths, a block twice in one of them, and own rows
    in a prefix's blocks: rows are read, so any may be named again."""
    c = Case([90, 64, 33], [0, 4, 7, 9], [9, 1, 0, 5, 16, 3, 8, 2, 1], 1, 2, 4, 128, 16, BF, seed=11)
    c.ptable[1] = c.ptable[0]
    c.ptable[2, 1] = c.ptable[2, 0]
    c.table[4] = c.ptable[0, 0]
    ws = c.ws()
    out, lse = c.call(ws)
    assert status(ws) == 0
    c.compare(out, lse)


@pytest.mark.parametrize("bits", [0, 8])
def test_queries_written_just_before(bits):
    """Captured with an append on one stream that writes the prefix's rows and the queries right before
    (kernels begin while those before them end), the two calls of a graph on one workspace: replayed with
    new inputs, the bits of calls with a synchronize between them."""
    N, H, G, d, bs, n = 6, 2, 4, 128, 16, 200
    pb = -(-n // bs)
    ptable = torch.arange(pb, dtype=torch.int32, device=DEV).view(1, pb)
    table = (pb + torch.arange(N, dtype=torch.int32, device=DEV)).view(N, 1)
    K = torch.zeros(pb + N, H, bs, d, dtype=BF, device=DEV)
    V = torch.zeros_like(K)
    plens = torch.tensor([n], dtype=torch.int32, device=DEV)
    lens = torch.full((N,), 3, dtype=torch.int32, device=DEV)
    plan = pkg.RopePlan(d)
    pk, pv = (torch.zeros(1, n, H, d, dtype=BF, device=DEV) for _ in range(2))
    nk, nv = (torch.zeros(N, 3, H, d, dtype=BF, device=DEV) for _ in range(2))
    q = torch.zeros(N, 3, H * G, d, dtype=BF, device=DEV)
    rq, one, two = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    ws = pkg.alloc_prefix_attention_workspace(q, H, bs, 1, pb * bs)
    cache = pkg.alloc_q8_cache(pb + N, H, bs, d, device=DEV)
    aws = pkg.alloc_attention_workspace(q, H, bs)

    def fill(seed):
        for i, x in enumerate((pk, pv, nk, nv, q)):
            x.copy_(rnd(x.shape, BF, 100 * seed + i))

    def run(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        if bits:
            pkg.rkv_q8_append(cache, nk, nv, table, lens, rope=plan, q=q, out_q=rq)
            pause()
            pkg.rkv_q8_attention(rq, cache, table, lens, out=one, workspace=aws)
            pause()
            K8, V8 = pkg.rkv_q8_read(cache, table, lens, 3)
            two[:, :, :H].copy_(K8.view(N, H, 3, d).transpose(1, 2))
            two[:, :, H:2 * H].copy_(V8.view(N, H, 3, d).transpose(1, 2))
            return
        pkg.rkv_paged_append(K, V, pk, pv, ptable, plens, rope=plan)
        pause()
        pkg.rkv_paged_append(K, V, nk, nv, table, lens, rope=plan, q=q, out_q=rq)
        pause()
        pkg.rkv_prefix_attention(rq, K, V, ptable, plens, table, lens, out=one, workspace=ws)
        pause()
        pkg.rkv_prefix_attention(one, K, V, ptable, plens, table, lens, out=two, workspace=ws)

    fill(0)
    run(True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(False)
    for seed in range(1, 9):
        fill(seed)
        run(True)
        torch.cuda.synchronize()
        want = [x.clone() for x in (one, two)]
        for x in (one, two, rq, K, V):
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one, want[0]) and torch.equal(two, want[1])


def test_two_graphs_on_one_workspace():
    """Two captured calls of other sizes share a workspace and are replayed in turn on one stream, without a
    wait between them: each call writes what it reads there."""
    a = Case([700], [0, 40], [12] * 40, 1, 2, 4, 128, 16, BF, seed=21)
    b = Case([130, 90], [0, 9, 20], [40] * 20, 2, 2, 4, 64, 32, BF, seed=22)
    cs = (a, b)
    plain = [c.call(c.ws())[0] for c in cs]
    ws = max((c.ws() for c in cs), key=lambda x: x.numel())
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    graphs, outs, held = [], [], []
    for c in cs:
        out = torch.zeros_like(c.q)
        args = (c.q, c.K, c.V, c.ptable.to(DEV), ints(c.plens), c.table.to(DEV), ints(c.lens))
        kw = dict(cu_seqs=ints(c.groups), out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.rkv_prefix_attention(*args, **kw)
        graphs.append(g)
        outs.append(out)
        held.append((args, kw))
    for _ in range(20):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], plain[0]) and torch.equal(outs[1], plain[1])


@pytest.mark.parametrize("dt, bs", [(FP, 16), (BF, 4), (BF, 16)], ids=["fp32", "bf16-b4", "bf16"])
@pytest.mark.parametrize("every", [2, 5])
def test_empty_prefixes_between_others(dt, bs, every):
    """Empty prefixes in turn with others, several of each a block, whose queries take one another's place in shared
    memory: call after call the bits of the first, and those of the definition."""
    P, S = 1200, 2400
    plens = [0 if p % every else 1 + p % 70 for p in range(P)]
    c = Case(plens, list(range(0, S + 1, 2)), [1 + s % 3 for s in range(S)], 1, 1, 2, 64, bs, dt, seed=31)
    ws = c.ws()
    out, lse = c.call(ws)
    for _ in range(10):
        again, lse2 = c.call(ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert status(ws) == 0
    c.K, c.V = c.K.cpu(), c.V.cpu()
    c.groups = list(range(0, 401, 2))
    for first in (0, P - 200):  # 200 prefixes at either end
        part = Case.__new__(Case)
        part.__dict__.update(c.__dict__)
        a, b = slice(first, first + 200), slice(2 * first, 2 * first + 400)
        part.plens, part.ptable, part.lens, part.table, part.q = c.plens[a], c.ptable[a], c.lens[b], c.table[b], c.q[b]
        part.compare(out[b], lse[b])


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
def test_one_workspace_while_sequences_end(dt):
    """A workspace made for the largest batch serves the batches after it: sequences and whole prefixes leave, and
    tiles and teams are chosen anew. The bits of calls with a workspace of their own; nothing behind it is written."""
    most = Case([700, 90, 400], [0, 100, 180, 257], [4 + s % 7 for s in range(257)], 2, 2, 4, 128, 16, dt, seed=41)
    n = most.ws().numel()
    room = torch.full((n + (1 << 20),), 0xa5, dtype=torch.uint8, device=DEV)
    for sizes in ([100, 80, 77], [100, 80, 76], [129], [128], [65, 0, 64], [64], [33], [32], [17, 16], [16], [5, 3, 2], [1]):
        c = Case.__new__(Case)
        c.__dict__.update(most.__dict__)
        S = sum(sizes)
        c.plens, c.ptable = most.plens[:len(sizes)], most.ptable[:len(sizes)]
        c.groups = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        c.lens, c.table, c.q = most.lens[:S], most.table[:S], most.q[:S].contiguous()
        room[:256] = 0
        out, lse = c.call(room[:n])
        assert status(room[:n]) == 0 and (room[n:] == 0xa5).all()
        own, lse2 = c.call()
        assert torch.equal(out, own) and torch.equal(lse, lse2)
        c.compare(out[:3], lse[:3], seqs=min(S, 3))
