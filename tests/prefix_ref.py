"""Attention over shared prefixes in 64 bits, with the quantities that
cache_ref.attention_bounds takes."""
from __future__ import annotations

import math

import torch


def group_of(groups, s):
    """The prefix of sequence s (None: none); groups: first sequence of each, and behind the last."""
    for p in range(len(groups) - 1):
        if groups[p] <= s < groups[p + 1]:
            return p
    return None


def rows_of(pool, table, lens):
    """Per line of the table [H, len, d] fp64."""
    out, bs = [], pool.shape[2]
    for s, n in enumerate(lens):
        n = max(n, 0)
        x = pool.cpu()[table[s, :-(-n // bs)].long().cpu()].double()
        out.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
    return out


def attention(q, prefix_k, prefix_v, groups, own_k, own_v, lens, scale):
    """(out, lse, A, L) as cache_ref.attention; prefix_*: per prefix, own_*: per
    sequence [H, rows, d] fp64."""
    S, T, Hq, d = q.shape
    out = torch.zeros(S, T, Hq, d, dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((S, T, Hq), -math.inf, dtype=torch.float64)
    L = torch.zeros(S, T, Hq, dtype=torch.float64)
    for s in range(S):
        H = own_k[s].shape[0]
        p = group_of(groups, s)
        for t in range(T):
            see = max(0, lens[s] - T + t + 1)
            k, v = own_k[s][:, :see], own_v[s][:, :see]
            if p is not None:
                k, v = torch.cat([prefix_k[p], k], 1), torch.cat([prefix_v[p], v], 1)
            if k.shape[1] == 0:
                continue
            qs = q[s, t].double().cpu().view(H, Hq // H, d)
            z = (qs @ k.mT) * scale
            le = torch.logsumexp(z, -1)
            w = torch.exp(z - le[..., None])
            out[s, t] = (w @ v).reshape(Hq, d)
            A[s, t] = (w @ v.abs()).reshape(Hq, d)
            lse[s, t] = le.reshape(-1)
            L[s, t] = (qs.abs() @ k.abs().mT).amax(-1).reshape(-1)
    return out, lse, A, L
