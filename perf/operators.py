"""The operators of a paged KV cache in use, as workloads: rotary positions, appending to the cache
(plain and at 4 bits) and attention over it.

`run` with `own` false computes each operator in elementary torch operations; with `own` true it makes
the calls a user makes of the library.  `exact` computes the same values in 64 bits from the
definitions.

Conventions shared by all cases: a sequence's rows live in blocks of a pool [blocks, heads, block, d]
named by a block table; `lens` counts a sequence's rows including the tokens the call brings; query
heads come in groups of `gqa` per KV head.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GROUP = 32  # values that share one 4-bit scale


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a batch: the new token's queries and keys, slices of a fused projection
        {"name": "rope-decode", "op": "rope", "tokens": 64, "heads": 32, "kv_heads": 8, "d": 128,
         "rot": 128, "pairs": "half", "scaling": "none", "dtype": "bf16", "inverse": False, "far": 16384},
        # a long prompt's chunk far beyond the trained length, half of each head rotated
        {"name": "rope-prompt", "op": "rope", "tokens": 16384, "heads": 40, "kv_heads": 8, "d": 128,
         "rot": 64, "pairs": "interleaved", "scaling": "by_parts", "dtype": "bf16", "inverse": False,
         "far": 131072},
        # the gradient of the rotation in a training step (fp32, an odd number of tokens)
        {"name": "rope-grad", "op": "rope", "tokens": 4097, "heads": 32, "kv_heads": 8, "d": 64,
         "rot": 64, "pairs": "half", "scaling": "linear", "dtype": "fp32", "inverse": True, "far": 32768},
        # one decode step of a batch of 64: one row each, positions apart from rows (compressed cache)
        {"name": "append-decode", "op": "append", "seqs": 64, "new": 1, "ragged": False, "gqa": 4,
         "kv_heads": 8, "d": 128, "rot": 128, "pairs": "half", "dtype": "bf16", "block": 16,
         "rows": 1152},
        # ragged prompts written into fresh caches
        {"name": "append-prompt", "op": "append", "seqs": 24, "new": 2111, "ragged": True, "gqa": 4,
         "kv_heads": 8, "d": 128, "rot": 128, "pairs": "half", "dtype": "bf16", "block": 128,
         "rows": 4224},
        # the same two at 4 bits, each followed by reading the written rows back
        {"name": "q4write-decode", "op": "q4write", "seqs": 64, "new": 1, "ragged": False, "gqa": 4,
         "kv_heads": 8, "d": 128, "rot": 128, "pairs": "half", "dtype": "bf16", "block": 16,
         "rows": 1152},
        {"name": "q4write-prompt", "op": "q4write", "seqs": 16, "new": 1766, "ragged": True, "gqa": 4,
         "kv_heads": 8, "d": 128, "rot": 0, "pairs": "half", "dtype": "bf16", "block": 64,
         "rows": 1766},
        # a single sequence just before its compression: latency
        {"name": "attn-one", "op": "attn", "seqs": 1, "new": 1, "gqa": 4, "kv_heads": 8, "d": 128,
         "dtype": "bf16", "block": 16, "rows": 1152, "least": 1152},
        # a batch of ragged sequences up to 4224 rows, five query heads a KV head
        {"name": "attn-batch", "op": "attn", "seqs": 64, "new": 1, "gqa": 5, "kv_heads": 8, "d": 128,
         "dtype": "bf16", "block": 128, "rows": 4224, "least": 131},
        # eight new tokens a sequence (drafted tokens checked in one pass, or an observation window)
        {"name": "attn-verify", "op": "attn", "seqs": 16, "new": 8, "gqa": 4, "kv_heads": 8, "d": 64,
         "dtype": "bf16", "block": 16, "rows": 16389, "least": 777},
        # one very long sequence at 4 bits, an odd number of rows
        {"name": "q4attn-one", "op": "q4attn", "seqs": 1, "new": 1, "gqa": 5, "kv_heads": 8, "d": 128,
         "dtype": "bf16", "block": 128, "rows": 131071, "least": 131071},
        # a batch at 4 bits
        {"name": "q4attn-batch", "op": "q4attn", "seqs": 64, "new": 1, "gqa": 4, "kv_heads": 8,
         "d": 128, "dtype": "bf16", "block": 16, "rows": 4224, "least": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "q4write", "attn", "q4attn"])
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    gqa = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    pairs = rng.choice(["half", "interleaved"])
    rot = rng.choice([d, d, d // 2, 32])
    if op == "rope":
        far = rng.choice([4096, 32768, 131072])
        return {"op": op, "tokens": _log(rng, 1, 16384 if dtype == "bf16" else 8192), "heads": min(gqa * kv, 32), "kv_heads": kv, "d": d,
                "rot": rot, "pairs": pairs, "scaling": rng.choice(["none", "linear", "ntk", "by_parts"]),
                "dtype": dtype, "inverse": rng.random() < 0.4, "far": far}
    if op in ("append", "q4write"):
        ragged = rng.random() < 0.5
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, min(2048, 8000 // seqs))) if ragged else rng.choice([1, 1, 2, 5])
        return {"op": op, "seqs": seqs, "new": new, "ragged": ragged, "gqa": min(gqa, 8), "kv_heads": kv, "d": d,
                "rot": rot if rng.random() < 0.8 else 0, "pairs": pairs, "dtype": dtype,
                "block": rng.choice([8, 16, 64, 128]), "rows": new + _log(rng, 1, 1500)}
    seqs = _log(rng, 1, 64)
    rows = _log(rng, 8, (60000 if op == "attn" else 120000) // seqs)
    return {"op": op, "seqs": seqs, "new": rng.choice([1, 1, 1, 2, 4, 8]) if gqa <= 8 else 1, "gqa": gqa,
            "kv_heads": kv, "d": d, "dtype": dtype if op == "attn" else "bf16",
            "block": rng.choice([8, 16, 32, 64, 128]), "rows": rows, "least": _log(rng, 1, rows)}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the largest among them, in a fixed irregular order."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _cpu_gen(seed):
    g = torch.Generator()
    g.manual_seed(int(seed) * 104729 + 7)
    return g


def _table(seqs, rows, block, seed):
    """A shuffled block table that covers `rows` rows of each sequence, and the pool's blocks."""
    nb = -(-rows // block)
    blocks = seqs * nb + 3
    perm = torch.randperm(blocks, generator=_cpu_gen(seed))[: seqs * nb]
    return perm.reshape(seqs, nb).to(torch.int32).to(DEV), blocks


def _rope_args(case):
    return {"rot_dim": case["rot"], "interleaved": case["pairs"] == "interleaved",
            "scaling": case.get("scaling", "none"), "base": 10000.0,
            "factor": 1.0 if case.get("scaling", "none") == "none" else 8.0, "original_len": 8192.0,
            "low": 1.0, "high": 4.0}


def _counts(case):
    """New tokens of each sequence."""
    if not case["ragged"]:
        return [case["new"]] * case["seqs"]
    return _spread(case["seqs"], max(1, case["new"] // 7), case["new"])


def _lens(case):
    return _spread(case["seqs"], min(case["least"], case["rows"]), case["rows"])


def prepare(case, seed):
    g = _gen(seed)
    op, d, H = case["op"], case["d"], case["kv_heads"]
    dt = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    st = {"case": dict(case)}
    if op == "rope":
        T, Hq = case["tokens"], case["heads"]
        qkv = rnd(T, (Hq + 2 * H) * d).to(dt)  # a fused projection: q and k are strided views
        st["q"] = qkv[:, : Hq * d].view(T, Hq, d)
        st["k"] = qkv[:, Hq * d: (Hq + H) * d].view(T, H, d)
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        st["out_q"] = torch.empty(T, Hq, d, dtype=dt, device=DEV)
        st["out_k"] = torch.empty(T, H, d, dtype=dt, device=DEV)
        if own:
            import decode_kv_cache_02_gb300 as pkg
            st["plan"] = pkg.RopePlan(**_rope_args(case))
        return st

    S, bs = case["seqs"], case["block"]
    st["table"], blocks = _table(S, case["rows"], bs, seed)
    if op in ("append", "q4write"):
        counts = _counts(case)
        total = sum(counts)
        # ragged prompts fill fresh caches; decode steps append behind older rows
        lens = counts if case["ragged"] else _spread(S, min(case["rows"], case["new"] + 1), case["rows"])
        Hq = case["gqa"] * H
        qkv = rnd(total, (Hq + 2 * H) * d)
        qkv[:, Hq * d:(Hq + H) * d] += rnd(H * d)  # keys carry a steady offset in each channel
        qkv = qkv.to(dt)
        st["q"] = qkv[:, : Hq * d].view(total, Hq, d)
        st["k"] = qkv[:, Hq * d:(Hq + H) * d].view(total, H, d)
        st["v"] = qkv[:, (Hq + H) * d:].view(total, H, d)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st["positions"] = torch.randint(0, 32768, (total,), generator=g, device=DEV, dtype=torch.int32)
        st["out_q"] = torch.empty(total, Hq, d, dtype=dt, device=DEV)
        if op == "append":
            st["K"] = torch.zeros(blocks, H, bs, d, dtype=dt, device=DEV)
            st["V"] = torch.zeros_like(st["K"])
        else:
            for n in ("K", "V"):
                st[n + "_codes"] = torch.zeros(blocks, H, bs, d // 2, dtype=torch.uint8, device=DEV)
                st[n + "_scales"] = torch.zeros(blocks, H, bs, d // GROUP, 2, dtype=torch.bfloat16, device=DEV)
            n_read = max(counts)
            st["n_read"] = n_read
            st["first"] = (st["lens"] - torch.tensor(counts, dtype=torch.int32, device=DEV)).to(torch.int32)
            st["K_rows"] = torch.zeros(S * H, n_read, d, dtype=torch.bfloat16, device=DEV)
            st["V_rows"] = torch.zeros_like(st["K_rows"])
        if own:
            import decode_kv_cache_02_gb300 as pkg
            st["plan"] = pkg.RopePlan(**_rope_args(case)) if case["rot"] else None
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
            if op == "q4write":
                st["cache"] = pkg.Q4Cache(st["K_codes"], st["K_scales"], st["V_codes"], st["V_scales"])
        return st

    # attention: keys with a steady offset in each channel, queries of ordinary size
    T, G = case["new"], case["gqa"]
    lens = torch.tensor(_lens(case), dtype=torch.int32)
    st["lens"] = lens[torch.randperm(S, generator=_cpu_gen(seed + 1))].to(DEV)
    st["q"] = rnd(S, T, H * G, d).to(dt)
    kshift = 0.5 * rnd(H, 1, d)
    if op == "attn":
        st["K"] = torch.empty(blocks, H, bs, d, dtype=dt, device=DEV)
        st["V"] = torch.empty_like(st["K"])
        st["K"].normal_(generator=g)
        st["K"] += kshift.to(dt)
        st["V"].normal_(generator=g)
    else:
        for n in ("K", "V"):
            shift = kshift if n == "K" else 0.0 * kshift
            parts = [_quantise(rnd(min(256, blocks - i), H, bs, d) + shift) for i in range(0, blocks, 256)]
            st[n + "_codes"], st[n + "_scales"] = (torch.cat(x) for x in zip(*parts))
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(S, T, H * G, dtype=torch.float32, device=DEV)
    st["rows"] = case["rows"]
    if own:
        import decode_kv_cache_02_gb300 as pkg
        if op == "attn":
            st["ws"] = pkg.alloc_attention_workspace(st["q"], H, case["rows"])
        else:
            st["cache"] = pkg.Q4Cache(st["K_codes"], st["K_scales"], st["V_codes"], st["V_scales"])
            st["ws"] = pkg.alloc_attention_workspace(st["q"], H, case["rows"])
    return st


# ------------------------------------------------------- plain torch forms --

def _freqs(a):
    """(angle per position of each pair, factor of the rotated values), 64 bits."""
    r = a["rot_dim"]
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    base = a["base"]
    if a["scaling"] == "ntk" and r > 2:
        base = base * a["factor"] ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if a["scaling"] == "linear":
        f = f / a["factor"]
    if a["scaling"] == "by_parts":
        turns = a["original_len"] * f / (2 * math.pi)
        keep = ((turns - a["low"]) / (a["high"] - a["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / a["factor"])
    return f


def _rotate(x, pos, a, inverse=False):
    """x [tokens, heads, d] rotated by its positions, in 32 bits (the angles in 64)."""
    x = x.float()
    r = a["rot_dim"]
    if r == 0:
        return x
    ang = pos.double()[:, None] * _freqs(a)
    c, s = ang.cos().float()[:, None], ang.sin().float()[:, None]
    if inverse:
        s = -s
    y = x.clone()
    if a["interleaved"]:
        e, o = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = e * c - o * s, o * c + e * s
    else:
        e, o = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = e * c - o * s, o * c + e * s
    return y


def _bf16_below(x):
    """The largest bf16 that is not above x (64 bits)."""
    y = x.to(torch.bfloat16)
    i = y.view(torch.int16)
    down = torch.where(y.float() > 0, i - 1, torch.where(y.float() < 0, i + 1, torch.full_like(i, -32767)))
    return torch.where(y.double() > x, down, i).view(torch.bfloat16)


def _quantise(x):
    """Codes and (scale, low) of fp32 rows [..., d]: groups of 32 values, low = the largest bf16 at or
    below the smallest value, scale = the smallest bf16 at or above (largest - low) / 15, code = the
    whole number nearest to (x - low) * r with r the fp32 nearest to 1 / scale.  Values next to a
    border between two codes are common (bf16 inputs on a bf16 grid), so this is done in 64 bits.
    Bytes are laid out so that 16 bits hold four neighbours of a group and a row's groups alternate."""
    d = x.shape[-1]
    xg = x.reshape(*x.shape[:-1], d // GROUP, GROUP).double()
    lo = _bf16_below(xg.amin(-1))
    s = -_bf16_below((lo.double() - xg.amax(-1)) / torch.full((1,), 15.0, dtype=torch.float64, device=x.device))
    r = torch.where(s > 0, 1.0 / s.double(), torch.zeros_like(s, dtype=torch.float64)).float().double()
    c = ((xg - lo.double()[..., None]) * r[..., None]).round().clamp(0, 15)
    c = c.to(torch.uint8).reshape(*x.shape[:-1], d // GROUP, 8, 4).transpose(-3, -2)
    b = c[..., 0::2] | (c[..., 1::2] << 4)
    return b.reshape(*x.shape[:-1], d // 2).contiguous(), torch.stack([s, lo], -1).contiguous()


def _values(codes, scales):
    """fp32 rows from codes [..., d / 2] and (scale, low) [..., d / 32, 2]."""
    n = scales.shape[-2]
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 8, n, 4).transpose(-3, -2)
    c = c.reshape(*codes.shape[:-1], n, GROUP).float()
    sc = scales.float()
    return (c * sc[..., 0:1] + sc[..., 1:2]).reshape(*codes.shape[:-1], n * GROUP)


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


def _attend(q, k, v, lens):
    """q [S, T, Hq, d], k and v [S, H, N, d] in 32 bits: (out, log of the sum of exponentials)."""
    S, T, Hq, d = q.shape
    H, N = k.shape[1], k.shape[2]
    G = Hq // H
    qf = q.float().view(S, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(S, H, T * G, d)
    z = torch.matmul(qf, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    t = torch.arange(T * G, device=DEV) // G
    last = lens.long()[:, None] - T + t  # the newest row each query sees
    seen = (torch.arange(N, device=DEV) <= last[..., None])[:, None]
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(N, device=DEV) < lens.long()[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log()).squeeze(-1)
    back = lambda x: x.view(S, H, T, G, -1).permute(0, 2, 1, 3, 4).reshape(S, T, Hq, -1)  # noqa: E731
    return back(o), back(lse[..., None]).squeeze(-1)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    a = _rope_args(case) if "rot" in case else None
    if op == "rope":
        dt = DTYPES[case["dtype"]]
        return (_rotate(st["q"], st["positions"], a, case["inverse"]).to(dt),
                _rotate(st["k"], st["positions"], a, case["inverse"]).to(dt))
    if op in ("append", "q4write"):
        blk, row = _slots(st)
        k = _rotate(st["k"], st["positions"], a)
        q = _rotate(st["q"], st["positions"], a).to(st["q"].dtype)
        if op == "append":
            st["K"][blk, :, row] = k.to(st["K"].dtype)
            st["V"][blk, :, row] = st["v"]
            return q, st["K"], st["V"]
        outs = [q]
        S, H, n, d = case["seqs"], case["kv_heads"], st["n_read"], case["d"]
        for name, x in (("K", k), ("V", st["v"].float())):
            c, s = _quantise(x)
            st[name + "_codes"][blk, :, row] = c
            st[name + "_scales"][blk, :, row] = s
            # read the new rows back
            r = st["first"].long()[:, None] + torch.arange(n, device=DEV)
            ok = r < st["lens"].long()[:, None]
            r = torch.where(ok, r, torch.zeros_like(r))
            b = st["table"].long().gather(1, r // case["block"])
            val = _values(st[name + "_codes"][b, :, r % case["block"]], st[name + "_scales"][b, :, r % case["block"]])
            val = val.permute(0, 2, 1, 3)  # [S, H, n, d]
            keep = st[name + "_rows"].view(S, H, n, d)
            keep.copy_(torch.where(ok[:, None, :, None], val.to(keep.dtype), keep))
            outs.append(st[name + "_rows"])
        return tuple(outs)
    if op == "attn":
        k, v = _gathered(st["K"], st["table"]).float(), _gathered(st["V"], st["table"]).float()
    else:
        k = _values(_gathered(st["K_codes"], st["table"]), _gathered(st["K_scales"], st["table"]))
        v = _values(_gathered(st["V_codes"], st["table"]), _gathered(st["V_scales"], st["table"]))
    o, lse = _attend(st["q"], k, v, st["lens"])
    return o.to(st["q"].dtype), lse


def _run_own(st):
    import decode_kv_cache_02_gb300 as pkg
    case = st["case"]
    op = case["op"]
    if op == "rope":
        return pkg.rkv_rope_apply(st["plan"], st["positions"], st["q"], st["k"], out_q=st["out_q"],
                                  out_k=st["out_k"], inverse=case["inverse"])
    if op in ("append", "q4write"):
        cu = st["cu"] if case["ragged"] else None
        rope = {} if st["plan"] is None else {"rope": st["plan"], "positions": st["positions"]}
        if op == "append":
            q = pkg.rkv_paged_append(st["K"], st["V"], st["k"], st["v"], st["table"], st["lens"], cu_tokens=cu,
                                     q=st["q"], out_q=st["out_q"], workspace=st["ws"], **rope)
            return q, st["K"], st["V"]
        q = pkg.rkv_q4_append(st["cache"], st["k"], st["v"], st["table"], st["lens"], cu_tokens=cu, q=st["q"],
                              out_q=st["out_q"], workspace=st["ws"], **rope)
        k, v = pkg.rkv_q4_read(st["cache"], st["table"], st["lens"], st["n_read"], first=st["first"],
                               out_K=st["K_rows"], out_V=st["V_rows"], workspace=st["ws"])
        return q, k, v
    if op == "attn":
        return pkg.rkv_paged_attention(st["q"], st["K"], st["V"], st["table"], st["lens"], max_rows=st["rows"],
                                       out=st["out"], lse=st["lse"], workspace=st["ws"])
    return pkg.rkv_q4_attention(st["q"], st["cache"], st["table"], st["lens"], max_rows=st["rows"],
                                out=st["out"], lse=st["lse"], workspace=st["ws"])


def run(st):
    return _run_own(st) if own else _run_plain(st)


def work(case):
    op, d, H = case["op"], case["d"], case["kv_heads"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["tokens"] * (case["heads"] + H)
        return {"bytes": 2 * e * n * d + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    row4 = d // 2 + 4 * (d // GROUP)
    if op in ("append", "q4write"):
        total, Hq = sum(_counts(case)), case["gqa"] * H
        q = 2 * e * total * Hq * d
        read, rows = 2 * e * total * H * d, 2 * total * H
        if op == "append":
            return {"bytes": q + read + rows * d * e, "flops": 3 * total * (Hq + H) * case["rot"]}
        # written at 4 bits, read again, and given back as rows
        return {"bytes": q + read + rows * (2 * row4 + 2 * d), "flops": 3 * total * (Hq + H) * case["rot"] + 6 * rows * d}
    total, T, G = sum(_lens(case)), case["new"], case["gqa"]
    row = d * e if op == "attn" else row4
    return {"bytes": 2 * total * H * row + 2 * e * case["seqs"] * T * H * G * d,
            "flops": 4 * total * H * T * G * d}


# ------------------------------------------------- the definitions, 64 bits --

def _turn64(x, pos, a, inverse):
    """Rotation in 64 bits, as complex products."""
    y = x.double().clone()
    r = a["rot_dim"]
    if r == 0:
        return y
    b = a["base"] * (a["factor"] ** (r / (r - 2.0)) if a["scaling"] == "ntk" and r > 2 else 1.0)
    f = []
    for i in range(r // 2):
        w = b ** (-2.0 * i / r)
        if a["scaling"] == "linear":
            w /= a["factor"]
        elif a["scaling"] == "by_parts":
            t = (a["original_len"] * w / (2 * math.pi) - a["low"]) / (a["high"] - a["low"])
            t = min(1.0, max(0.0, t))
            w = t * w + (1 - t) * w / a["factor"]
        f.append(w)
    ang = torch.outer(pos.double(), torch.tensor(f, dtype=torch.float64, device=DEV))
    if inverse:
        ang = -ang
    u = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    if a["interleaved"]:
        z = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * u
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., : r // 2].contiguous(), y[..., r // 2: r].contiguous()) * u
        y[..., : r // 2], y[..., r // 2: r] = z.real, z.imag
    return y


def _floor8(x):
    """x rounded down to 8 significant bits (64-bit arithmetic)."""
    m, e = torch.frexp(x)
    return torch.floor(m * 256.0) / 256.0 * torch.exp2(e.double())


def _through4(x):
    """What 4 bits keep of fp64 rows [..., d]."""
    g = x.unflatten(-1, (-1, GROUP))
    low = _floor8(g.min(-1, keepdim=True).values)
    fifteen = torch.full_like(low, 15.0)
    step = -_floor8((low - g.max(-1, keepdim=True).values) / fifteen)
    per = (fifteen / 15 / torch.where(step > 0, step, fifteen)).float().double()
    c = torch.where(step > 0, torch.round((g - low) * per), torch.zeros_like(g))
    return (low + step * c.clamp(0, 15)).flatten(-2)


def _attend64(st, case):
    S, T, H, G, d, bs = case["seqs"], case["new"], case["kv_heads"], case["gqa"], case["d"], case["block"]
    out = torch.zeros(S, T, H * G, d, dtype=torch.float64, device=DEV)
    lse = torch.full((S, T, H * G), -math.inf, dtype=torch.float64, device=DEV)
    n_of = st["lens"].tolist()
    for s in range(S):
        n = n_of[s]
        ids = st["table"][s, : -(-n // bs)].long()
        side = []
        for name in ("K", "V"):
            if case["op"] == "attn":
                x = st[name][ids].double()
            else:
                by = st[name + "_codes"][ids].int()
                sc = st[name + "_scales"][ids].double()
                w = by[..., 0::2] + 256 * by[..., 1::2]  # 16 bits: four codes of one group
                w = w.unflatten(-1, (8, d // GROUP))
                c = torch.stack([(w >> (4 * i)) & 15 for i in range(4)], -1).double()  # [.., 8, groups, 4]
                c = c.movedim(-2, -3).flatten(-2)  # [.., groups, 32]
                x = (c * sc[..., :1] + sc[..., 1:]).flatten(-2)
            side.append(x.movedim(1, 0).flatten(1, 2)[:, :n])  # [H, n, d]
        k, v = side
        for t in range(T):
            see = n - T + t + 1
            if see <= 0:
                continue
            qs = st["q"][s, t].double().view(H, G, d)
            z = qs @ k[:, :see].mT / d ** 0.5
            le = torch.logsumexp(z, -1)
            out[s, t] = (torch.exp(z - le[..., None]) @ v[:, :see]).reshape(H * G, d)
            lse[s, t] = le.reshape(-1)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("attn", "q4attn"):
        return _attend64(st, case)
    a = _rope_args(case)
    if op == "rope":
        return (_turn64(st["q"], st["positions"], a, case["inverse"]),
                _turn64(st["k"], st["positions"], a, case["inverse"]))
    q, k = _turn64(st["q"], st["positions"], a, False), _turn64(st["k"], st["positions"], a, False)
    counts, lens = _counts(case), st["lens"].tolist()
    v = st["v"].double()
    if op == "append":
        outs = [q]
        for pool, x in ((st["K"], k), (st["V"], v)):
            y, j = pool.double(), 0
            for s, c in enumerate(counts):
                rows = torch.arange(lens[s] - c, lens[s], device=DEV)
                y[st["table"][s].long()[rows // case["block"]], :, rows % case["block"]] = x[j: j + c]
                j += c
            outs.append(y)
        return tuple(outs)
    outs = [q]
    for x in (k, v):
        y = torch.zeros(case["seqs"], case["kv_heads"], st["n_read"], case["d"], dtype=torch.float64, device=DEV)
        z, j = _through4(x), 0
        for s, c in enumerate(counts):
            y[s, :, :c] = z[j: j + c].movedim(1, 0)
            j += c
        outs.append(y.flatten(0, 1))
    return tuple(outs)
