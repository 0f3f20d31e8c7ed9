"""More operators of a paged KV cache in use, as workloads: attention of a batch whose sequences share
long prefixes, and a cache held in 8 bits (append, read back, attention).

`run` with `own` false computes each operator in elementary torch operations; with `own` true it makes
the calls a user makes of the library.  `exact` computes the same values in 64 bits from the
definitions.

Conventions shared by all cases: a sequence's own rows live in blocks of a pool [blocks, heads, block, d]
named by a block table; `lens` counts them including the tokens the call brings; query heads come in
groups of `gqa` per KV head.  A shared prefix is rows of the same pool, named by a table of its own:
every token of its sequences sees all of them, before the sequence's own rows.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a handful of samples of one prompt, just begun: latency
        {"name": "prefix-small", "op": "prefix", "prefixes": 1, "seqs": 4, "alone": 0, "new": 1, "gqa": 4, "kv_heads": 8,
         "d": 128, "dtype": "bf16", "block": 16, "prefix_rows": 1024, "prefix_least": 1024, "rows": 40, "least": 33},
        # the rollouts of one prompt, each with a compressed cache of its own
        {"name": "prefix-rollouts", "op": "prefix", "prefixes": 1, "seqs": 64, "alone": 0, "new": 1, "gqa": 4, "kv_heads": 8,
         "d": 128, "dtype": "bf16", "block": 128, "prefix_rows": 8192, "prefix_least": 8192, "rows": 1152, "least": 131},
        # a training batch: eight prompts with several samples each, some requests of other users beside them
        {"name": "prefix-prompts", "op": "prefix", "prefixes": 8, "seqs": 131, "alone": 3, "new": 1, "gqa": 5, "kv_heads": 8,
         "d": 128, "dtype": "bf16", "block": 16, "prefix_rows": 4224, "prefix_least": 517, "rows": 1152, "least": 257},
        # many samples over one very long document, an odd number of rows
        {"name": "prefix-long", "op": "prefix", "prefixes": 1, "seqs": 128, "alone": 0, "new": 1, "gqa": 4, "kv_heads": 8,
         "d": 128, "dtype": "bf16", "block": 128, "prefix_rows": 131071, "prefix_least": 131071, "rows": 128, "least": 9},
        # eight drafted tokens a sequence checked in one pass
        {"name": "prefix-verify", "op": "prefix", "prefixes": 2, "seqs": 16, "alone": 0, "new": 8, "gqa": 4, "kv_heads": 8,
         "d": 64, "dtype": "bf16", "block": 16, "prefix_rows": 16389, "prefix_least": 9001, "rows": 640, "least": 77},
        # a fp32 cache (a numerics check of a rollout)
        {"name": "prefix-fp32", "op": "prefix", "prefixes": 2, "seqs": 24, "alone": 0, "new": 1, "gqa": 4, "kv_heads": 4,
         "d": 128, "dtype": "fp32", "block": 64, "prefix_rows": 2049, "prefix_least": 1500, "rows": 300, "least": 20},
        # one decode step of a batch of 64 written at 8 bits and read back
        {"name": "q8write-decode", "op": "q8write", "seqs": 64, "new": 1, "ragged": False, "gqa": 4, "kv_heads": 8,
         "d": 128, "rot": 128, "pairs": "half", "dtype": "bf16", "block": 16, "rows": 1152},
        # ragged prompts written into fresh caches at 8 bits and read back for their compression
        {"name": "q8write-prompt", "op": "q8write", "seqs": 16, "new": 1766, "ragged": True, "gqa": 4, "kv_heads": 8,
         "d": 128, "rot": 128, "pairs": "half", "dtype": "bf16", "block": 64, "rows": 1766},
        # a single sequence just before its compression: latency
        {"name": "q8attn-one", "op": "q8attn", "seqs": 1, "new": 1, "gqa": 4, "kv_heads": 8, "d": 128, "dtype": "bf16",
         "block": 16, "rows": 1152, "least": 1152},
        # a batch of ragged sequences up to 4224 rows, five query heads a KV head
        {"name": "q8attn-batch", "op": "q8attn", "seqs": 64, "new": 1, "gqa": 5, "kv_heads": 8, "d": 128, "dtype": "bf16",
         "block": 128, "rows": 4224, "least": 131},
        # one very long sequence, an odd number of rows
        {"name": "q8attn-long", "op": "q8attn", "seqs": 1, "new": 1, "gqa": 8, "kv_heads": 8, "d": 128, "dtype": "bf16",
         "block": 16, "rows": 131071, "least": 131071},
        # eight new tokens a sequence
        {"name": "q8attn-verify", "op": "q8attn", "seqs": 16, "new": 8, "gqa": 4, "kv_heads": 8, "d": 64, "dtype": "bf16",
         "block": 16, "rows": 16389, "least": 777},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "q8write", "q8attn", "q8attn"])
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    gqa = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    if op == "q8write":
        ragged = rng.random() < 0.5
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, min(2048, 8000 // seqs))) if ragged else rng.choice([1, 1, 2, 5])
        rot = rng.choice([d, d, d // 2, 32, 0])
        return {"op": op, "seqs": seqs, "new": new, "ragged": ragged, "gqa": min(gqa, 8), "kv_heads": kv, "d": d, "rot": rot,
                "pairs": rng.choice(["half", "interleaved"]), "dtype": dtype, "block": rng.choice([8, 16, 64, 128]),
                "rows": new + _log(rng, 1, 1500)}
    if op == "q8attn":
        seqs = _log(rng, 1, 64)
        rows = _log(rng, 8, 120000 // seqs)
        return {"op": op, "seqs": seqs, "new": rng.choice([1, 1, 1, 2, 4, 8]) if gqa <= 8 else 1, "gqa": gqa, "kv_heads": kv,
                "d": d, "dtype": "bf16", "block": rng.choice([8, 16, 32, 64, 128]), "rows": rows, "least": _log(rng, 1, rows)}
    prefixes = rng.choice([1, 1, 1, 2, 3, 5, 8])
    seqs = prefixes * _log(rng, 1, 96 // prefixes) + rng.choice([0, 0, 1, 3])
    new = rng.choice([1, 1, 1, 2, 5]) if gqa <= 8 else 1
    queries = seqs * new * gqa * kv
    # a bound on the work: the prefixes' products, and the rows that fp32 would copy
    most = min(100000 // prefixes, int(1.6e8 if dtype == "bf16" else 6e6) // queries + 64)
    rows = _log(rng, 1, 40000 // seqs)
    prefix_rows = _log(rng, 16, max(17, most))
    return {"op": op, "prefixes": prefixes, "seqs": seqs, "alone": rng.choice([0, 0, 0, 1, seqs // 3]), "new": new, "gqa": gqa,
            "kv_heads": kv, "d": d, "dtype": dtype, "block": rng.choice([8, 16, 32, 64, 128]), "prefix_rows": prefix_rows,
            "prefix_least": _log(rng, 1, prefix_rows), "rows": max(rows, new), "least": _log(rng, 1, max(rows, new))}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _cpu_gen(seed):
    g = torch.Generator()
    g.manual_seed(int(seed) * 104729 + 7)
    return g


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the largest among them, in a fixed irregular order."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _tables(counts, seed):
    """Shuffled block tables [n, blocks each] for each (n, blocks each), and the pool's blocks."""
    total = sum(n * nb for n, nb in counts)
    perm = torch.randperm(total + 3, generator=_cpu_gen(seed))
    out, at = [], 0
    for n, nb in counts:
        out.append(perm[at: at + n * nb].reshape(n, nb).to(torch.int32).to(DEV))
        at += n * nb
    return out, total + 3


def _groups(case):
    """First sequence of each prefix, and behind the last; the sequences past it have no prefix."""
    shared, P = case["seqs"] - case["alone"], case["prefixes"]
    return [shared * p // P for p in range(P + 1)]


def _counts(case):
    """New tokens of each sequence."""
    if not case["ragged"]:
        return [case["new"]] * case["seqs"]
    return _spread(case["seqs"], max(1, case["new"] // 7), case["new"])


def _lens(case):
    return _spread(case["seqs"], min(case["least"], case["rows"]), case["rows"])


def _prefix_lens(case):
    return _spread(case["prefixes"], min(case["prefix_least"], case["prefix_rows"]), case["prefix_rows"])


def _rope_args(case):
    return {"rot_dim": case["rot"], "interleaved": case["pairs"] == "interleaved", "base": 10000.0}


def prepare(case, seed):
    g = _gen(seed)
    op, d, H, S, bs = case["op"], case["d"], case["kv_heads"], case["seqs"], case["block"]
    dt = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    st = {"case": dict(case)}
    if own:
        import decode_kv_cache_02_gb300 as pkg
    if op == "q8write":
        (st["table"],), blocks = _tables([(S, -(-case["rows"] // bs))], seed)
        counts = _counts(case)
        total = sum(counts)
        # ragged prompts fill fresh caches; decode steps append behind older rows
        lens = counts if case["ragged"] else _spread(S, min(case["rows"], case["new"] + 1), case["rows"])
        Hq = case["gqa"] * H
        qkv = rnd(total, (Hq + 2 * H) * d)
        qkv[:, Hq * d:(Hq + H) * d] += rnd(H * d)  # keys carry a steady offset in each channel
        qkv = qkv.to(dt)
        st["q"] = qkv[:, : Hq * d].view(total, Hq, d)  # slices of a fused projection
        st["k"] = qkv[:, Hq * d:(Hq + H) * d].view(total, H, d)
        st["v"] = qkv[:, (Hq + H) * d:].view(total, H, d)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st["positions"] = torch.randint(0, 32768, (total,), generator=g, device=DEV, dtype=torch.int32)
        st["out_q"] = torch.empty(total, Hq, d, dtype=dt, device=DEV)
        for n in ("K", "V"):
            st[n + "_codes"] = torch.zeros(blocks, H, bs, d, dtype=torch.int8, device=DEV)
            st[n + "_scales"] = torch.zeros(blocks, H, bs, dtype=torch.float32, device=DEV)
        st["n_read"] = max(counts)
        st["first"] = (st["lens"] - torch.tensor(counts, dtype=torch.int32, device=DEV)).to(torch.int32)
        st["K_rows"] = torch.zeros(S * H, st["n_read"], d, dtype=torch.bfloat16, device=DEV)
        st["V_rows"] = torch.zeros_like(st["K_rows"])
        if own:
            st["plan"] = pkg.RopePlan(**_rope_args(case)) if case["rot"] else None
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
            st["cache"] = pkg.Q8Cache(st["K_codes"], st["K_scales"], st["V_codes"], st["V_scales"])
        return st

    # attention: keys with a steady offset in each channel, queries of ordinary size
    T, G = case["new"], case["gqa"]
    lens = torch.tensor(_lens(case), dtype=torch.int32)
    st["lens"] = lens[torch.randperm(S, generator=_cpu_gen(seed + 1))].to(DEV)
    st["q"] = rnd(S, T, H * G, d).to(dt)
    kshift = 0.5 * rnd(H, 1, d)
    if op == "prefix":
        (st["table"], st["prefix_table"]), blocks = _tables(
            [(S, -(-case["rows"] // bs)), (case["prefixes"], -(-case["prefix_rows"] // bs))], seed)
        st["groups"] = _groups(case)
        st["cu"] = torch.tensor(st["groups"], dtype=torch.int32, device=DEV)
        st["prefix_lens"] = torch.tensor(_prefix_lens(case), dtype=torch.int32, device=DEV)
        st["K"] = torch.empty(blocks, H, bs, d, dtype=dt, device=DEV)
        st["V"] = torch.empty_like(st["K"])
        st["K"].normal_(generator=g)
        st["K"] += kshift.to(dt)
        st["V"].normal_(generator=g)
    else:
        (st["table"],), blocks = _tables([(S, -(-case["rows"] // bs))], seed)
        for n in ("K", "V"):
            shift = kshift if n == "K" else 0.0 * kshift
            parts = [_quantise(rnd(min(512, blocks - i), H, bs, d) + shift) for i in range(0, blocks, 512)]
            st[n + "_codes"], st[n + "_scales"] = (torch.cat(x) for x in zip(*parts))
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(S, T, H * G, dtype=torch.float32, device=DEV)
    if own and op == "prefix":
        st["ws"] = pkg.alloc_prefix_attention_workspace(st["q"], H, case["rows"], case["prefixes"], case["prefix_rows"])
    elif own:
        st["cache"] = pkg.Q8Cache(st["K_codes"], st["K_scales"], st["V_codes"], st["V_scales"])
        st["ws"] = pkg.alloc_attention_workspace(st["q"], H, case["rows"])
    return st


# ------------------------------------------------------- plain torch forms --

def _rotate(x, pos, a):
    """x [tokens, heads, d] rotated by its positions, in 32 bits (the angles in 64)."""
    x = x.float()
    r = a["rot_dim"]
    if r == 0:
        return x
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    ang = pos.double()[:, None] * a["base"] ** (-2.0 * i / r)
    c, s = ang.cos().float()[:, None], ang.sin().float()[:, None]
    y = x.clone()
    if a["interleaved"]:
        e, o = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = e * c - o * s, o * c + e * s
    else:
        e, o = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = e * c - o * s, o * c + e * s
    return y


def _quantise(x):
    """Codes and scale of fp32 rows [..., d]: scale = the fp32 nearest to the largest magnitude / 127, code =
    the whole number nearest to x * r with r the fp32 nearest to 1 / scale.  Values next to a border between
    two codes are common (bf16 inputs on a bf16 grid), so this is done in 64 bits."""
    x = x.double()
    scale = (x.abs().amax(-1) / torch.full((1,), 127.0, dtype=torch.float64, device=x.device)).float()
    s = scale.double()
    r = torch.where(s >= 2.0 ** -126, 1.0 / s, torch.zeros_like(s)).float().double()
    return (x * r[..., None]).round().to(torch.int8), scale


def _slots(st):
    """(block, row in the block) of each new token."""
    cu, lens, bs = st["cu"].long(), st["lens"].long(), st["case"]["block"]
    total = st["k"].shape[0]
    j = torch.arange(total, device=DEV)
    s = torch.searchsorted(cu[1:].contiguous(), j, right=True)
    row = lens[s] - (cu[s + 1] - cu[s]) + (j - cu[s])
    return st["table"].long()[s, row // bs], row % bs


def _gathered(pool, table):
    """The rows of each sequence, [seqs, heads, rows, ...]."""
    x = pool[table.long()]  # [S, nb, H, bs, ...]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _sums(q, k, v, seen):
    """Largest logit m, sum of exp(z - m) and that of exp(z - m) v; q [B, H, M, d], k and v [B, H, N, d], 32 bits."""
    z = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(q.shape[-1]))
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _own_sums(q, k, v, lens):
    """_sums over each sequence's own rows; q [S, T, Hq, d]."""
    S, T, Hq, d = q.shape
    H, N = k.shape[1], k.shape[2]
    G = Hq // H
    qf = q.float().view(S, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(S, H, T * G, d)
    t = torch.arange(T * G, device=DEV) // G
    last = lens.long()[:, None] - T + t  # the newest row each query sees
    j = torch.arange(N, device=DEV)
    seen = (j <= last[..., None])[:, None]
    v = torch.where((j < lens.long()[:, None])[:, None, :, None], v, torch.zeros_like(v))
    return qf, _sums(qf, k, v, seen)


def _finish(parts, S, T, H, G):
    """(out, log of the sum of exponentials) [S, T, Hq, ..] of one or two (m, l, o) [S, H, T * G, ..]."""
    m = parts[0][0]
    for x in parts[1:]:
        m = torch.maximum(m, x[0])
    at = torch.where(m > -math.inf, m, torch.zeros_like(m))
    f = [torch.exp(x[0] - at) for x in parts]
    total = sum(x[1] * y for x, y in zip(parts, f))
    o = sum(x[2] * y for x, y in zip(parts, f)) / torch.where(total > 0, total, torch.ones_like(total))
    back = lambda x: x.view(S, H, T, G, -1).permute(0, 2, 1, 3, 4).reshape(S, T, H * G, -1)  # noqa: E731
    return back(o), back(m + total.log()).squeeze(-1)


def _run_plain(st):
    case = st["case"]
    op, S, H, d = case["op"], case["seqs"], case["kv_heads"], case["d"]
    if op == "q8write":
        a = _rope_args(case)
        blk, row = _slots(st)
        k = _rotate(st["k"], st["positions"], a)
        outs = [_rotate(st["q"], st["positions"], a).to(st["q"].dtype)]
        n = st["n_read"]
        r = st["first"].long()[:, None] + torch.arange(n, device=DEV)
        ok = r < st["lens"].long()[:, None]
        r = torch.where(ok, r, torch.zeros_like(r))
        b = st["table"].long().gather(1, r // case["block"])
        for name, x in (("K", k), ("V", st["v"].float())):
            c, s = _quantise(x)
            st[name + "_codes"][blk, :, row] = c
            st[name + "_scales"][blk, :, row] = s
            # read the new rows back
            val = st[name + "_codes"][b, :, r % case["block"]].float() * st[name + "_scales"][b, :, r % case["block"]][..., None]
            val = val.permute(0, 2, 1, 3)  # [S, H, n, d]
            keep = st[name + "_rows"].view(S, H, n, d)
            keep.copy_(torch.where(ok[:, None, :, None], val.to(keep.dtype), keep))
            outs.append(st[name + "_rows"])
        return tuple(outs)
    T, G = case["new"], case["gqa"]
    if op == "q8attn":
        k, v = (_gathered(st[n + "_codes"], st["table"]).float() * _gathered(st[n + "_scales"], st["table"])[..., None]
                for n in ("K", "V"))
        o, lse = _finish([_own_sums(st["q"], k, v, st["lens"])[1]], S, T, H, G)
        return o.to(st["q"].dtype), lse
    k, v = _gathered(st["K"], st["table"]).float(), _gathered(st["V"], st["table"]).float()
    qf, part = _own_sums(st["q"], k, v, st["lens"])
    first = [torch.full_like(part[0], -math.inf), torch.zeros_like(part[1]), torch.zeros_like(part[2])]
    for p in range(case["prefixes"]):
        a, b = st["groups"][p], st["groups"][p + 1]
        if a == b:
            continue
        k, v = (_gathered(st[n], st["prefix_table"][p: p + 1]).float() for n in ("K", "V"))
        seen = torch.arange(k.shape[2], device=DEV) < st["prefix_lens"][p]
        v = torch.where(seen[:, None], v, torch.zeros_like(v))
        qs = qf[a:b].transpose(0, 1).reshape(1, H, (b - a) * T * G, d)
        for x, y in zip(first, _sums(qs, k, v, seen)):
            x[a:b] = y.view(H, b - a, T * G, -1).transpose(0, 1)
    o, lse = _finish([first, part], S, T, H, G)
    return o.to(st["q"].dtype), lse


def _run_own(st):
    import decode_kv_cache_02_gb300 as pkg
    case = st["case"]
    if case["op"] == "q8write":
        cu = st["cu"] if case["ragged"] else None
        rope = {} if st["plan"] is None else {"rope": st["plan"], "positions": st["positions"]}
        q = pkg.rkv_q8_append(st["cache"], st["k"], st["v"], st["table"], st["lens"], cu_tokens=cu, q=st["q"],
                              out_q=st["out_q"], workspace=st["ws"], **rope)
        k, v = pkg.rkv_q8_read(st["cache"], st["table"], st["lens"], st["n_read"], first=st["first"],
                               out_K=st["K_rows"], out_V=st["V_rows"], workspace=st["ws"])
        return q, k, v
    if case["op"] == "q8attn":
        return pkg.rkv_q8_attention(st["q"], st["cache"], st["table"], st["lens"], max_rows=case["rows"],
                                    out=st["out"], lse=st["lse"], workspace=st["ws"])
    return pkg.rkv_prefix_attention(st["q"], st["K"], st["V"], st["prefix_table"], st["prefix_lens"], st["table"],
                                    st["lens"], cu_seqs=st["cu"], max_prefix_rows=case["prefix_rows"],
                                    max_rows=case["rows"], out=st["out"], lse=st["lse"], workspace=st["ws"])


def run(st):
    return _run_own(st) if own else _run_plain(st)


def work(case):
    op, d, H, G = case["op"], case["d"], case["kv_heads"], case["gqa"]
    e = 2 if case["dtype"] == "bf16" else 4
    row8 = d + 4
    if op == "q8write":
        total = sum(_counts(case))
        # written at 8 bits, read again, and given back as rows
        return {"bytes": 2 * e * total * G * H * d + 2 * total * H * (e * d + 2 * row8 + 2 * d),
                "flops": 3 * total * (G * H + H) * case["rot"] + 6 * total * H * d}
    T, S = case["new"], case["seqs"]
    own_rows = sum(_lens(case))
    flops = 4 * own_rows * H * T * G * d
    moved = 2 * own_rows * H * (row8 if op == "q8attn" else d * e) + 2 * e * S * T * H * G * d
    if op == "prefix":
        first = _groups(case)
        for p, n in enumerate(_prefix_lens(case)):
            if first[p + 1] > first[p]:
                moved += 2 * n * H * d * e
                flops += 4 * n * (first[p + 1] - first[p]) * T * G * H * d
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------- the definitions, 64 bits --

def _turn64(x, pos, a):
    """Rotation in 64 bits, as complex products."""
    y = x.double().clone()
    r = a["rot_dim"]
    if r == 0:
        return y
    w = torch.tensor([a["base"] ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device=DEV)
    ang = torch.outer(pos.double(), w)
    u = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    if a["interleaved"]:
        z = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * u
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., : r // 2].contiguous(), y[..., r // 2: r].contiguous()) * u
        y[..., : r // 2], y[..., r // 2: r] = z.real, z.imag
    return y


def _through8(x):
    """What 8 bits keep of fp64 rows [..., d]: whole steps of the row's largest magnitude over 127."""
    step = (x.abs().max(-1, keepdim=True).values.div(127.0)).float()
    per = step.double().clamp(min=2.0 ** -126).reciprocal().float().double()
    return torch.round(x * per) * step.double()


def _heads64(values, ids, n):
    """The first n rows of the blocks `ids` of a pool, [H, n, d] in 64 bits."""
    x = values(ids.long()).movedim(1, 0)
    return x.flatten(1, 2)[:, :n]


def _attend64(st, case):
    S, T, H, G, d, bs = case["seqs"], case["new"], case["kv_heads"], case["gqa"], case["d"], case["block"]
    out = torch.zeros(S, T, H * G, d, dtype=torch.float64, device=DEV)
    lse = torch.full((S, T, H * G), -math.inf, dtype=torch.float64, device=DEV)
    if case["op"] == "q8attn":
        pools = [lambda i, n=n: st[n + "_codes"][i].double() * st[n + "_scales"][i].double()[..., None] for n in "KV"]
        of = [None] * S
    else:
        pools = [lambda i, n=n: st[n][i].double() for n in "KV"]
        of = [next((p for p in range(case["prefixes"]) if st["groups"][p] <= s < st["groups"][p + 1]), None) for s in range(S)]
    n_of = st["lens"].tolist()
    shared, held = None, None
    for s in range(S):
        rows = [_heads64(x, st["table"][s, : -(-n_of[s] // bs)], n_of[s]) for x in pools]
        before = 0
        if of[s] is not None:
            if held != of[s]:
                n = int(st["prefix_lens"][of[s]])
                shared = [_heads64(x, st["prefix_table"][of[s], : -(-n // bs)], n) for x in pools]
                held = of[s]
            before = shared[0].shape[1]
        for t in range(T):
            see = max(0, n_of[s] - T + t + 1)
            if before + see == 0:
                continue
            qs = st["q"][s, t].double().view(H, G, d)
            z = qs @ rows[0][:, :see].mT / d ** 0.5
            if before:
                z = torch.cat([qs @ shared[0].mT / d ** 0.5, z], -1)
            le = torch.logsumexp(z, -1)
            w = torch.exp(z - le[..., None])
            o = w[..., before:] @ rows[1][:, :see]
            if before:
                o = o + w[..., :before] @ shared[1]
            out[s, t] = o.reshape(H * G, d)
            lse[s, t] = le.reshape(-1)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "q8write":
        return _attend64(st, case)
    a = _rope_args(case)
    q, k = _turn64(st["q"], st["positions"], a), _turn64(st["k"], st["positions"], a)
    outs = [q]
    for x in (k, st["v"].double()):
        y = torch.zeros(case["seqs"], case["kv_heads"], st["n_read"], case["d"], dtype=torch.float64, device=DEV)
        z, j = _through8(x), 0
        for s, c in enumerate(_counts(case)):
            y[s, :, :c] = z[j: j + c].movedim(1, 0)
            j += c
        outs.append(y.flatten(0, 1))
    return tuple(outs)
