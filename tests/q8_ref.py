"""The 8-bit cache in 64 bits: what a row of head_dim values is stored as."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def quantise(x):
    """(codes int8, scale fp32) of fp64 rows [..., d] that hold fp32 values: scale
    the fp32 nearest to the largest magnitude / 127 (the quotient in 64 bits is
    never so near the middle of two fp32 that its own rounding matters: 24 bits
    over 7), r the fp32 nearest to 1 / scale, codes the whole numbers nearest to
    x * r (48 bits: exact in 64), halves to even.  A row with a NaN or an
    infinity: scale NaN, codes 0."""
    top = x.abs().amax(-1)
    good = torch.isfinite(x).all(-1)
    scale = torch.where(good, top / 127, torch.full_like(top, float("nan"))).float()
    s = scale.double()
    r = torch.where(s >= 2.0 ** -126, 1 / s, torch.zeros_like(s)).float().double()
    c = torch.round(torch.where(good[..., None], x, torch.zeros_like(x)) * r.nan_to_num(0.0)[..., None])
    return c.to(torch.int8), scale


def rows_of(codes, scales, table, lens):
    """Per sequence [H, len, d] fp64 of a pool's codes and scales."""
    out, bs = [], codes.shape[2]
    for s, n in enumerate(lens):
        ids = table[s, :-(-max(n, 0) // bs)].long().cpu()
        x = codes.cpu()[ids].double() * scales.cpu()[ids].double()[..., None]
        out.append(x.transpose(0, 1).flatten(1, 2)[:, :max(n, 0)])
    return out
