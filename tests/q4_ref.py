"""Attention over 4-bit rows in 64 bits, and how far the kernel may be from it.

With P_j the softmax's weights and a group's values s (c - 8) + (low + 8 s):

- a weight is off by delta: the logit is a sum of d products and 2 d / 32 group
  terms in fp32, off by at most (d + 40) 2^-24 of sum |q| (15 s + |low|) (the
  sums of q over a group have 32 terms), its scaling by 4 * 2^-24 of itself,
  and the exponential's argument, at most |lse| and the range of the
  reference (below 130) away from zero, by 2^-24 of itself, the exponential by 2
  ulp.  Numerator and denominator: 2 delta sum P |v|.
- P s is rounded to fp16, half a step 2^-11, or, below 2^-14 beside a reference
  of 2^11 or more, to steps of 2^-24: a row is then off by 2^-25 * 8 where
  its group's largest row is at 2^2 or more (a group at most 2^-8 of its row's
  largest, and that a factor 2 below its power of two, else the product takes
  two bf16 parts, 2^-16): N 2^-24 max_j P_j g_j with g_j = max(s, |low|).
- the weights of (scale, low) are taken as two bf16 parts, 2^-16, or, with more
  than 16 queries a KV head, as one, half a step 2^-8; they meet low + 8 s.
- sums in fp32 over a warp's quarter of the rows, and their joins: each step off
  by 2^-23 (the tensor core's additions may cut), (rows / 2 + 128) 2^-24 of
  sum P (s |c - 8| + |low| + 8 s).
- the output's rounding: 2^-8 (bf16).
"""
from __future__ import annotations

import math

import torch

from tests import cache_ref as ref

U16, U32, UH = ref.U16, ref.U32, 2.0 ** -11


def rows_of(codes, scales, table, lens):
    """Per sequence (c [H, n, W, 32], s [H, n, W], low [H, n, W]), fp64."""
    out = []
    bs = codes.shape[2]
    for s, n in enumerate(lens):
        ids = table[s, :-(-max(n, 0) // bs)].long().cpu()
        c, sc, lo = ref.unpack(codes.cpu()[ids], scales.cpu()[ids])  # [nb, H, bs, W, 32] ..
        out.append(tuple(x.transpose(0, 1).flatten(1, 2)[:, :n] for x in (c, sc, lo)))
    return out


def attention(q, K, V, lens, scale):
    """q [S, T, Hq, d] against K, V of rows_of: (out, lse, |out| bound, lse bound)."""
    S, T, Hq, d = q.shape
    out = torch.zeros(S, T, Hq, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse = torch.full((S, T, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for s in range(S):
        H = K[s][0].shape[0]
        G = Hq // H
        for t in range(T):
            see = lens[s] - T + t + 1
            if see <= 0:
                continue
            (kc, ks, kl), (vc, vs, vl) = (tuple(x[:, :see] for x in y[s]) for y in (K, V))
            flat = lambda x: x.flatten(-2)  # noqa: E731
            wide = lambda x: x[..., None].expand(*x.shape, 32).flatten(-2)  # noqa: E731
            k = flat(kc * ks[..., None] + kl[..., None])
            qs = q[s, t].double().cpu().view(H, G, d)
            z = qs @ k.mT * scale
            le = torch.logsumexp(z, -1)
            P = torch.exp(z - le[..., None])
            v = flat(vc * vs[..., None] + vl[..., None])
            o = P @ v
            mag = (qs.abs() @ wide(15 * ks + kl.abs()).mT).amax(-1)
            delta = mag * (d + 40) * U32 * abs(scale) + z.abs().amax(-1) * 4 * U32 + \
                (3 * le.abs() + 200) * U32
            codes = wide(vs) * flat((vc - 8).abs())
            b = 2 * delta[..., None] * (P @ v.abs())
            b = b + UH * (P @ codes)
            g = wide(torch.maximum(vs, vl.abs()))  # [H, see, d]
            b = b + see * 2.0 ** -24 * (P[..., None] * g[:, None]).amax(2)
            b = b + (U16 if T * G > 16 else 2.0 ** -16) * (P @ wide((vl + 8 * vs).abs()))
            b = b + (see / 2 + 128) * U32 * (P @ (codes + wide(vl.abs() + 8 * vs)))
            b = b + U16 * (o.abs() + b) + 1e-37
            out[s, t], bound[s, t] = o.reshape(Hq, d), b.reshape(Hq, d)
            lse[s, t] = le.reshape(-1)
            lb[s, t] = (delta + (see / 4 + 16) * U32 + 4 * U32 * le.abs()).reshape(-1)
    return out, lse, bound, lb


def check(q, cache, table, lens, scale, out, lse):
    """The worst |error| / bound of a call; asserts that it is at most 1."""
    K = rows_of(cache.K_codes, cache.K_scales, table, lens)
    V = rows_of(cache.V_codes, cache.V_scales, table, lens)
    e, el, b, lb = attention(q, K, V, lens, scale)
    got = out.double().cpu()
    hidden = torch.isinf(el)
    assert torch.equal(hidden, torch.isinf(lse.cpu())) and (got[hidden] == 0).all()
    assert torch.isfinite(got).all()
    worst = float(((got - e).abs() / b.clamp(min=1e-37))[~hidden].max()) if (~hidden).any() else 0.0
    assert worst <= 1, worst
    dl = (lse.double().cpu() - el).abs()[~hidden]
    assert (dl <= lb[~hidden]).all(), float((dl / lb[~hidden]).max())
    return worst
