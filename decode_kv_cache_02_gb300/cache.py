"""ctypes binding of the cache in use (include/rkv.h, "the cache in use"): one
function per C entry point with the same name.

As in ``rkv``: tensor metadata is checked here, outputs the caller did not pass
are allocated, raw pointers and the stream go to the library, and there is no
fallback.  Calls run on the device of their tensors and, unless ``stream`` is
given, on that device's current stream.

These calls run for every layer of every token, and a decode step's kernels
take a few microseconds, so the common case (tensors on the current device, the
current stream) takes no context manager, and descriptors are packed bytes.

``rkv_rope_apply`` takes part in autograd.  The other calls have no gradient:
what they write or return carries no history, whatever their inputs require.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import rkv as _rkv
from .rkv import RKV_DTYPE_BF16, RKV_DTYPE_FP32, _Q4Cache, _RopeConfig, _RopePlan, _check

RKV_MAX_NEW_TOKENS = 64
_MAX_ROWS = 1 << 30  # of a sequence in an attention (past 31 bits an int would wrap on its way to C)
_DTYPE = {torch.bfloat16: RKV_DTYPE_BF16, torch.float32: RKV_DTYPE_FP32}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_pack_rows = struct.Struct("@Pqqq").pack      # rkv_rows
_pack_desc = struct.Struct("@q7i4x").pack     # rkv_paged_desc
_pack_q4 = struct.Struct("@4P").pack          # rkv_q4_cache
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def load():
    return _rkv._lib or _rkv.load()  # without the lock once it is there


def _elsewhere(fn, t: torch.Tensor, stream, *args, **kw):
    """fn on another stream, or on tensors of another device than the current
    one: what it allocates belongs to that stream."""
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is not None and stream.device != t.device:
        raise ValueError("stream and tensors must be on one device")
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)


def _away(t: torch.Tensor, stream) -> bool:
    return stream is not None or not t.is_cuda or t.get_device() != _current_device()


def _ints(t, name: str, dev: int, *shape) -> int:
    """The address of a contiguous int32 tensor."""
    if t.dtype != _I32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t.data_ptr()


def _token_ints(t, name: str, dev: int, tokens: int) -> int:
    if t.dtype != _I32 or t.numel() != tokens or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32, one per token")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t.data_ptr()


def _dtype(t: torch.Tensor) -> int:
    c = _DTYPE.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")
    return c


def _rows(t, name: str, dev: int, heads, d: int, dtype, tokens: int, per_seq: int) -> bytes:
    """The rows of [tokens, heads, d] or [seqs, per_seq, heads, d], strides as
    they are, as an rkv_rows."""
    st = t.stride()
    if len(st) == 3:
        tok, head, one = st
        seq = per_seq * tok
        ok = t.shape == (tokens, heads, d)
    elif len(st) == 4:
        seq, tok, head, one = st
        ok = t.shape == (tokens // per_seq if per_seq else t.shape[0], per_seq, heads, d)
    else:
        ok, one = False, 1
    if not ok or one != 1 or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} [{tokens}, {heads}, {d}] or [{tokens // max(per_seq, 1)}, "
                         f"{per_seq}, {heads}, {d}] with a contiguous last dimension")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return _pack_rows(t.data_ptr(), seq, tok, head)


def _workspace(ws, dev: int):
    """(address, bytes) of a workspace; its error word needs 256 bytes."""
    if ws is None:
        return None, 0
    n = ws.numel()
    if ws.dtype != _U8 or n < 256 or not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor of at least 256 bytes on the "
                         "device of the other tensors")
    return ws.data_ptr(), n


# ------------------------------------------------------------------ rotary --

class RopePlan:
    """Rotary positions (rkv_rope_config in include/rkv.h): pairs (i, i +
    rot_dim/2) of a head, or with ``interleaved`` (2i, 2i + 1), turned by pos *
    base^(-2i/rot_dim); ``scaling`` "none", "linear" (``factor``), "ntk"
    (``factor``) or "by_parts" (``factor``, ``original_len``, ``low``,
    ``high``).  ``freqs`` gives the rot_dim/2 angles per position instead of
    base and scaling.  The turned values are multiplied by ``attn_factor``."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                 low: float = 1.0, high: float = 32.0, attn_factor: float = 1.0, freqs=None):
        if scaling not in _SCALING:
            raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
        c = _RopePlan()
        if freqs is not None:
            f = [float(x) for x in freqs]
            if 2 * len(f) != int(rot_dim):
                raise ValueError("freqs must hold rot_dim / 2 angles")
            arr = (ctypes.c_double * max(len(f), 1))(*f)
            rc = load().rkv_rope_init_freqs(int(rot_dim), 1 if interleaved else 0, arr,
                                            float(attn_factor), ctypes.byref(c))
            _check(rc, "rkv_rope_init_freqs")
        else:
            cfg = _RopeConfig(int(rot_dim), 1 if interleaved else 0, _SCALING[scaling], float(base),
                              float(factor), float(original_len), float(low), float(high),
                              float(attn_factor))
            _check(load().rkv_rope_init(ctypes.byref(cfg), ctypes.byref(c)), "rkv_rope_init")
        self._c = c
        self._packed = bytes(c)
        self.rot_dim = int(rot_dim)


def _aligned(g):
    """A gradient as rows the library takes (autograd hands out expanded ones)."""
    if g.numel() == 0:
        return g.new_empty(g.shape)
    unit = 16 // g.element_size()
    st = g.stride()
    if st[-1] != 1 or any(x % unit for x in st[:-1]):
        g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone(memory_format=torch.contiguous_format)


class _Rotation(torch.autograd.Function):
    """rkv_rope_apply with its gradient, which turns back (and has the same)."""

    @staticmethod
    def forward(ctx, rope, positions, inverse, q, k):
        ctx.set_materialize_grads(False)
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(positions)
        out = rkv_rope_apply(rope, positions, q, k, inverse=inverse)
        if k is not None and not q.requires_grad:
            ctx.mark_non_differentiable(out[0])
        elif k is not None and not k.requires_grad:
            ctx.mark_non_differentiable(out[1])
        return out

    @staticmethod
    def backward(ctx, gq, gk=None):
        positions, = ctx.saved_tensors
        gs = [_aligned(g) for g in (gq, gk) if g is not None]
        if not gs:
            return None, None, None, None, None
        out = rkv_rope_apply(ctx.rope, positions, *gs, inverse=not ctx.inverse)
        out = list(out) if len(gs) == 2 else [out]
        return (None, None, None, None if gq is None else out.pop(0),
                None if gk is None else out.pop(0))


def rkv_rope_apply(rope: RopePlan, positions, q, k=None, out_q=None, out_k=None,
                   inverse: bool = False, stream=None):
    """q (and k) [tokens, heads, d] or [seqs, n, heads, d] turned by positions
    (int32, one per token); inverse=True turns back, the map of the gradients.
    Outputs may be the inputs.  Returns out_q, or (out_q, out_k) with k.

    Takes part in autograd where q or k requires a gradient (to q and k);
    outputs of the caller's own are refused then (torch.no_grad() allows them)."""
    if _away(q, stream):
        return _elsewhere(rkv_rope_apply, q, stream, rope, positions, q, k, out_q, out_k, inverse)
    if (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        if out_q is not None or out_k is not None:
            raise ValueError("out_q and out_k take no gradient: leave them out, or call under "
                             "torch.no_grad()")
        return _Rotation.apply(rope, positions, bool(inverse), q, k)
    dev = q.get_device()
    sh = q.shape
    if len(sh) == 3:
        tokens, hq, d = sh
        per = tokens
    elif len(sh) == 4:
        seqs, per, hq, d = sh
        tokens = seqs * per
    else:
        raise ValueError("q must be [tokens, heads, d] or [seqs, n, heads, d]")
    dt, code = q.dtype, _dtype(q)
    if out_q is None:
        out_q = torch.empty(sh, dtype=dt, device=q.device)
    rk = rko = None
    hk = 0
    if k is not None:
        hk = k.shape[-2] if k.dim() > 1 else 0
        if out_k is None:
            out_k = torch.empty(k.shape, dtype=dt, device=q.device)
        rk = _rows(k, "k", dev, hk, d, dt, tokens, per)
        rko = _rows(out_k, "out_k", dev, hk, d, dt, tokens, per)
    elif out_k is not None:
        raise ValueError("out_k without k")
    rc = load().rkv_rope_apply(rope._packed, code, d, tokens, per or 1,
                               _token_ints(positions, "positions", dev, tokens),
                               1 if inverse else 0, hq, _rows(q, "q", dev, hq, d, dt, tokens, per),
                               _rows(out_q, "out_q", dev, hq, d, dt, tokens, per), hk, rk, rko,
                               _raw_stream(dev))
    if rc:
        _check(rc, "rkv_rope_apply")
    return out_q if k is None else (out_q, out_k)


# ------------------------------------------------------------------ append --

def _append(call, where, cache_args, dev, shape, k, v, block_table, lens, cu_tokens, rope,
            positions, q, out_q, workspace):
    nb, H, bs, d = shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
    S, mb = block_table.shape
    dims = k.dim()
    if dims == 3:
        tokens = k.shape[0]
    elif dims == 4:
        tokens = k.shape[0] * k.shape[1]
    else:
        raise ValueError("k must be [tokens, H, d] or [seqs, n, H, d]")
    cu = pos = None
    new = 0
    if cu_tokens is not None:
        if dims != 3:
            raise ValueError("with cu_tokens, tokens are numbered through: k [tokens, H, d]")
        cu = _ints(cu_tokens, "cu_tokens", dev, S + 1)
        per = tokens
    else:
        if tokens and (S == 0 or tokens % S):
            raise ValueError("without cu_tokens every sequence brings the same number of tokens")
        per = new = tokens // S if S else 0
    if positions is not None:
        if rope is None:
            raise ValueError("positions without a rope")
        pos = _token_ints(positions, "positions", dev, tokens)
    dt, code = k.dtype, _dtype(k)
    rq = ro = None
    G = 1
    if q is not None:
        hq = q.shape[-2] if q.dim() > 1 else 0
        G = hq // H if H else 0
        if G == 0 or G * H != hq:
            raise ValueError("the heads of q must be a multiple of the KV heads")
        if out_q is None:
            out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rq = _rows(q, "q", dev, hq, d, dt, tokens, per)
        ro = rq if out_q is q else _rows(out_q, "out_q", dev, hq, d, dt, tokens, per)
    elif out_q is not None:
        raise ValueError("out_q without q")
    rc = call(_pack_desc(S, H, G, d, bs, nb, mb, code), None if rope is None else rope._packed,
              *cache_args, _ints(block_table, "block_table", dev, S, mb),
              _ints(lens, "lens", dev, S), tokens, new, cu, pos,
              _rows(k, "k", dev, H, d, dt, tokens, per), _rows(v, "v", dev, H, d, dt, tokens, per),
              rq, ro, _workspace(workspace, dev)[0], _raw_stream(dev))
    if rc:
        _check(rc, where)
    return out_q


def _pools(K_pool, V_pool, dev: int):
    """The pools' common shape."""
    sh = K_pool.shape
    if len(sh) != 4 or V_pool.shape != sh or V_pool.dtype != K_pool.dtype \
            or not K_pool.is_contiguous() or not V_pool.is_contiguous() \
            or V_pool.get_device() != dev:
        raise ValueError("K_pool, V_pool must be contiguous [num_blocks, H, block_size, head_dim] "
                         "of one dtype on one device")
    return sh


def rkv_paged_append(K_pool, V_pool, k, v, block_table, lens, cu_tokens=None,
                     rope: RopePlan | None = None, positions=None, q=None, out_q=None,
                     workspace=None, stream=None):
    """Writes the new tokens' keys (turned by rope) and values into a paged
    cache; lens [S] counts the rows with the new tokens.  k, v [tokens, H, d]
    (cu_tokens [S + 1]: sequence s brings tokens cu[s] .. cu[s + 1] - 1;
    without, every sequence the same number) or [S, n, H, d].  positions
    default to the rows written.  q is turned (without a rope: copied) into
    out_q, which is returned (None without q)."""
    if _away(K_pool, stream):
        return _elsewhere(rkv_paged_append, K_pool, stream, K_pool, V_pool, k, v, block_table,
                          lens, cu_tokens, rope, positions, q, out_q, workspace)
    dev = K_pool.get_device()
    shape = _pools(K_pool, V_pool, dev)
    if k.dtype != K_pool.dtype:
        raise ValueError("k, v and the pools must share a dtype")
    return _append(load().rkv_paged_append, "rkv_paged_append",
                   (K_pool.data_ptr(), V_pool.data_ptr()), dev, shape, k, v, block_table, lens,
                   cu_tokens, rope, positions, q, out_q, workspace)


# ------------------------------------------------------------------ 4 bits --

class Q4Cache:
    """A paged cache held in 4 bits (rkv_q4_cache in include/rkv.h): codes
    uint8 [num_blocks, H, block_size, d / 2], scales bf16 [num_blocks, H,
    block_size, d / 32, 2] (scale, low), for K and for V."""

    def __init__(self, K_codes, K_scales, V_codes, V_scales):
        for t, n in ((K_codes, "K_codes"), (V_codes, "V_codes")):
            if t.dtype != _U8 or t.dim() != 4 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{n} must be contiguous CUDA uint8 [num_blocks, H, block_size, d/2]")
        nb, H, bs, half = K_codes.shape
        for t, n in ((K_scales, "K_scales"), (V_scales, "V_scales")):
            if t.dtype != torch.bfloat16 or half % 16 or not t.is_contiguous() \
                    or t.shape != (nb, H, bs, half // 16, 2):
                raise ValueError(f"{n} must be contiguous bf16 [num_blocks, H, block_size, d/32, 2]")
        if V_codes.shape != K_codes.shape:
            raise ValueError("K_codes and V_codes must have one shape")
        if any(t.device != K_codes.device for t in (K_scales, V_codes, V_scales)):
            raise ValueError("the arrays must be on one device")
        self.K_codes, self.K_scales, self.V_codes, self.V_scales = (K_codes, K_scales, V_codes,
                                                                    V_scales)
        self.shape = (nb, H, bs, 2 * half)
        self._c = _Q4Cache(K_codes.data_ptr(), K_scales.data_ptr(), V_codes.data_ptr(),
                           V_scales.data_ptr())
        self._packed = bytes(self._c)


def alloc_q4_cache(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int,
                   device="cuda") -> Q4Cache:
    """A zeroed 4-bit cache (5 bits a value with its scales)."""
    t = []
    for _ in range(2):
        t.append(torch.zeros((num_blocks, num_kv_heads, block_size, head_dim // 2), dtype=_U8,
                             device=device))
        t.append(torch.zeros((num_blocks, num_kv_heads, block_size, head_dim // 32, 2),
                             dtype=torch.bfloat16, device=device))
    return Q4Cache(*t)


def rkv_q4_append(cache: Q4Cache, k, v, block_table, lens, cu_tokens=None,
                  rope: RopePlan | None = None, positions=None, q=None, out_q=None,
                  workspace=None, stream=None):
    """rkv_paged_append into a 4-bit cache (k, v, q bf16 or fp32)."""
    at = cache.K_codes
    if _away(at, stream):
        return _elsewhere(rkv_q4_append, at, stream, cache, k, v, block_table, lens, cu_tokens,
                          rope, positions, q, out_q, workspace)
    return _append(load().rkv_q4_append, "rkv_q4_append", (cache._packed,), at.get_device(),
                   cache.shape, k, v, block_table, lens, cu_tokens, rope, positions, q, out_q,
                   workspace)


def rkv_q4_read(cache: Q4Cache, block_table, lens, n_rows: int, first=None, out_K=None,
                out_V=None, dtype=torch.bfloat16, workspace=None, stream=None):
    """(K, V) rows first[s] .. first[s] + n_rows - 1 of every sequence (first
    None: from row 0) as values [S * H, n_rows, d], the layout of rkv_score and
    rkv_compress.  Rows at or past lens[s] are not written (zeros where the
    output is allocated here)."""
    at = cache.K_codes
    if _away(at, stream):
        return _elsewhere(rkv_q4_read, at, stream, cache, block_table, lens, n_rows, first, out_K,
                          out_V, dtype, workspace)
    dev = at.get_device()
    nb, H, bs, d = cache.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
    S, mb = block_table.shape
    n_rows = int(n_rows)
    shape = (S * H, n_rows, d)
    if out_K is None:
        out_K = torch.zeros(shape, dtype=dtype if out_V is None else out_V.dtype, device=at.device)
    dt, code = out_K.dtype, _dtype(out_K)
    if out_V is None:
        out_V = torch.zeros(shape, dtype=dt, device=at.device)
    for t, n in ((out_K, "out_K"), (out_V, "out_V")):
        if t.shape != shape or t.dtype != dt or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{n} must be contiguous {list(shape)}, K and V of one dtype, on the "
                             "cache's device")
    rc = load().rkv_q4_read(_pack_desc(S, H, 1, d, bs, nb, mb, code), cache._packed,
                            _ints(block_table, "block_table", dev, S, mb),
                            _ints(lens, "lens", dev, S),
                            None if first is None else _ints(first, "first", dev, S), n_rows,
                            out_K.data_ptr(), out_V.data_ptr(), _workspace(workspace, dev)[0],
                            _raw_stream(dev))
    if rc:
        _check(rc, "rkv_q4_read")
    return out_K, out_V


# --------------------------------------------------------------- attention --

def rkv_attention_workspace_size(q, num_kv_heads: int, max_rows: int) -> int:
    """Workspace bytes of rkv_paged_attention and rkv_q4_attention for q [S,
    n_new, heads, d] over at most max_rows rows a sequence, on q's device."""
    if q.is_cuda and q.get_device() != _current_device():
        with torch.cuda.device(q.device):
            return rkv_attention_workspace_size(q, num_kv_heads, max_rows)
    H = int(num_kv_heads)
    if q.dim() != 4 or H < 1 or q.shape[2] == 0 or q.shape[2] % H:
        raise ValueError("q must be [num_seqs, n_new, H * gqa_group, d]")
    S, T, hq, d = q.shape
    if not 0 < max_rows <= _MAX_ROWS:
        raise ValueError("max_rows must be 1 .. 2^30")
    desc = _pack_desc(S, H, hq // H, d, 1, 1, int(max_rows), _dtype(q))
    n = int(load().rkv_attention_workspace_size(desc, T, int(max_rows)))
    if n == 0:
        raise ValueError("invalid workspace request")
    return n


def alloc_attention_workspace(q, num_kv_heads: int, max_rows: int) -> torch.Tensor:
    """A zero-filled uint8 tensor of rkv_attention_workspace_size() bytes."""
    return torch.zeros(rkv_attention_workspace_size(q, num_kv_heads, max_rows), dtype=_U8,
                       device=q.device)


def _attention(call, where, cache_args, dev, shape, q, block_table, lens, max_rows, scale, out,
               lse, workspace):
    nb, H, bs, d = shape
    sh = q.shape
    if len(sh) != 4:
        raise ValueError("q must be [num_seqs, n_new, H * gqa_group, d]")
    S, T, hq, _ = sh
    G = hq // H if H else 0
    if G == 0 or G * H != hq:
        raise ValueError("the heads of q must be a multiple of the KV heads")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
    mb = block_table.shape[1]
    dt = q.dtype
    max_rows = mb * bs if max_rows is None else int(max_rows)
    if not 0 < max_rows <= _MAX_ROWS:
        raise ValueError("max_rows (by default the table's rows) must be 1 .. 2^30")
    if out is None:
        out = torch.empty(sh, dtype=dt, device=q.device)
    at = None
    if lse is True:
        lse = torch.empty((S, T, hq), dtype=_F32, device=q.device)
    elif lse is False:
        lse = None
    if lse is not None:
        if lse.dtype != _F32 or lse.shape != (S, T, hq) or not lse.is_contiguous() \
                or lse.get_device() != dev:
            raise ValueError("lse must be contiguous fp32 [num_seqs, n_new, heads] on the device of "
                             "the other tensors")
        at = lse.data_ptr()
    desc = _pack_desc(S, H, G, d, bs, nb, mb, _dtype(q))
    if workspace is None:
        n = load().rkv_attention_workspace_size(desc, T, max_rows)
        workspace = torch.empty(max(n, 256), dtype=_U8, device=q.device)
    wp, wn = _workspace(workspace, dev)
    tokens = S * T
    rc = call(desc, T, _rows(q, "q", dev, hq, d, dt, tokens, T), *cache_args,
              _ints(block_table, "block_table", dev, S, mb), _ints(lens, "lens", dev, S), max_rows,
              1.0 / math.sqrt(d) if scale is None else scale,
              _rows(out, "out", dev, hq, d, dt, tokens, T), at, wp, wn, _raw_stream(dev))
    if rc:
        _check(rc, where)
    return out if lse is None else (out, lse)


def rkv_paged_attention(q, K_pool, V_pool, block_table, lens, max_rows: int | None = None,
                        scale: float | None = None, out=None, lse=None, workspace=None,
                        stream=None):
    """Attention of the newest tokens q [S, n_new, H * G, d] over a paged
    cache: token t of sequence s sees rows 0 .. lens[s] - n_new + t.  max_rows
    bounds lens (default: the table's rows; a tighter bound balances the work
    better), scale defaults to 1 / sqrt(d).  Returns out [S, n_new, H * G, d],
    or (out, lse) when lse is True or an fp32 tensor [S, n_new, H * G].
    Without a workspace (rkv_attention_workspace_size) scratch is allocated
    and device errors are not reported."""
    if _away(K_pool, stream):
        return _elsewhere(rkv_paged_attention, K_pool, stream, q, K_pool, V_pool, block_table,
                          lens, max_rows, scale, out, lse, workspace)
    dev = K_pool.get_device()
    shape = _pools(K_pool, V_pool, dev)
    if q.dtype != K_pool.dtype:
        raise ValueError("q and the pools must share a dtype")
    return _attention(load().rkv_paged_attention, "rkv_paged_attention",
                      (K_pool.data_ptr(), V_pool.data_ptr()), dev, shape, q, block_table, lens,
                      max_rows, scale, out, lse, workspace)


def rkv_q4_attention(q, cache: Q4Cache, block_table, lens, max_rows: int | None = None,
                     scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """rkv_paged_attention over a 4-bit cache (q bf16)."""
    at = cache.K_codes
    if _away(at, stream):
        return _elsewhere(rkv_q4_attention, at, stream, q, cache, block_table, lens, max_rows,
                          scale, out, lse, workspace)
    return _attention(load().rkv_q4_attention, "rkv_q4_attention", (cache._packed,),
                      at.get_device(), cache.shape, q, block_table, lens, max_rows, scale, out,
                      lse, workspace)
