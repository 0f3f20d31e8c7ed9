"""Plain 64-bit forms of the paged cache in use (rotary positions, appends,
4-bit groups, attention), and the bounds the tests hold the kernels to.

A rounding to a type is off by at most half a step, eps / 2 relative: bf16
2^-8, fp32 2^-24.
"""
from __future__ import annotations

import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def freqs(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            g = (original_len * f / (2 * math.pi) - low) / (high - low)
            g = min(1.0, max(0.0, g))
            f = f * g + f * (1 - g) / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, pos, f, interleaved=False, m=1.0, inverse=False):
    """fp64 rows x [tokens, heads, d] turned by pos * f (rot = 2 len(f))."""
    x = x.double().cpu().clone()
    rot = 2 * len(f)
    if rot == 0:
        return x
    a = pos.double().cpu()[:, None] * f[None]
    if inverse:
        a = -a
    c, s = torch.cos(a)[:, None] * m, torch.sin(a)[:, None] * m
    if interleaved:
        u, v = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
        x[..., 0:rot:2], x[..., 1:rot:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., : rot // 2].clone(), x[..., rot // 2: rot].clone()
        x[..., : rot // 2], x[..., rot // 2: rot] = u * c - v * s, v * c + u * s
    return x


def rotate_bound(x, y, rot, interleaved, dtype, m=1.0):
    """|error| allowed for y = rotate(x) computed in fp32 and rounded to dtype.

    The phase is cut to 2^-32 of a turn (below 2^-29), sine and cosine are
    within 2 ulp (2^-23 at most), the factor, the two products and the sum round
    once each: below 6 * 2^-24 times (|x| + |x'|); 8 leaves room for the plan's
    own rounding at far positions."""
    x = x.double().cpu().abs()
    s = x.clone()
    if rot:
        if interleaved:
            both = x[..., 0:rot:2] + x[..., 1:rot:2]
            s[..., 0:rot:2] = both
            s[..., 1:rot:2] = both
        else:
            both = x[..., : rot // 2] + x[..., rot // 2: rot]
            s[..., : rot // 2] = both
            s[..., rot // 2: rot] = both
    b = 8 * U32 * s * abs(m)
    if dtype == torch.bfloat16:
        b = b + U16 * (y.abs() + b)
    return b


# ------------------------------------------------------------------ 4 bits --

def floor_bf16(x):
    """x (fp64) rounded down to 8 significant bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.floor(m * 256) / 256, e)


def quantise(x):
    """(codes, scale, low) of fp64 rows [..., d], groups of 32."""
    g = x.unflatten(-1, (-1, 32))
    low = floor_bf16(g.min(-1).values)
    scale = -floor_bf16((low - g.max(-1).values) / 15)
    r = torch.where(scale > 0, 1 / torch.where(scale > 0, scale, torch.ones_like(scale)),
                    torch.zeros_like(scale)).float().double()
    c = torch.round((g - low[..., None]) * r[..., None])
    return c, scale, low


def unpack(codes, scales):
    """(codes, scale, low) as fp64 from the library's arrays."""
    W = scales.shape[-2]
    b = codes.cpu().to(torch.int64)
    w = (b[..., 0::2] | (b[..., 1::2] << 8)).unflatten(-1, (8, W))  # [.., 8, W] 16-bit words
    c = torch.stack([(w >> (4 * i)) & 15 for i in range(4)], -1)    # [.., 8, W, 4]
    c = c.transpose(-3, -2).flatten(-2).double()                    # [.., W, 32]
    sc = scales.cpu().double()
    return c, sc[..., 0], sc[..., 1]


def values(codes, scales):
    c, s, lo = unpack(codes, scales)
    return (c * s[..., None] + lo[..., None]).flatten(-2)


# --------------------------------------------------------------- attention --

def attention(q, rows_k, rows_v, lens, scale):
    """q [S, T, Hq, d]; rows_k, rows_v: per sequence [H, len, d] fp64.  Returns
    (out, lse, A, L): A = sum p |v| / sum p, L = the largest |q| |k| sum of a
    visible row, for the bounds."""
    S, T, Hq, d = q.shape
    out = torch.zeros(S, T, Hq, d, dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((S, T, Hq), -math.inf, dtype=torch.float64)
    L = torch.zeros(S, T, Hq, dtype=torch.float64)
    for s in range(S):
        H = rows_k[s].shape[0]
        G = Hq // H
        for t in range(T):
            see = lens[s] - T + t + 1
            if see <= 0:
                continue
            k, v = rows_k[s][:, :see], rows_v[s][:, :see]
            qs = q[s, t].double().cpu().view(H, G, d)
            z = (qs @ k.mT) * scale
            le = torch.logsumexp(z, -1)
            p = torch.exp(z - le[..., None])
            out[s, t] = (p @ v).reshape(Hq, d)
            A[s, t] = (p @ v.abs()).reshape(Hq, d)
            lse[s, t] = le.reshape(-1)
            L[s, t] = (qs.abs() @ k.abs().mT).amax(-1).reshape(-1)
    return out, lse, A, L


def attention_bounds(out, lse, A, L, scale, d, rows, kind, extra=0.0, extra_v=0.0):
    """(|out| bound, lse bound).

    Logits: a sum of d products in fp32, off by at most (d + 4) 2^-24 of the
    sum of magnitudes (and `extra`, what a format's offsets add); ex2 within 2
    ulp and the scale's rounding: delta.  A relative error of p shifts the
    mean by at most 2 delta A.  The probabilities' rounding to bf16 adds 2^-8
    A (`extra_v`: what the offsets add there); accumulation in fp32 over a
    warp's share of the rows and the join (rows / 4 + 64) 2^-24 A; the output's
    rounding 2^-8 |out| (bf16)."""
    scale = abs(scale)
    delta = (L * (d + 4) * U32 + extra) * scale + (lse.abs().nan_to_num(0, 0, 0) + 8) * 4 * U32
    b = (2 * delta[..., None] + (rows / 4 + 64) * U32) * A + extra_v + 1e-30
    if kind != "fp32":
        b = b + U16 * A
        b = b + U16 * (out.abs() + b)
    return b, delta + 8 * U32 * (1 + lse.abs().nan_to_num(0, 0, 0)) + rows / 4 * U32
