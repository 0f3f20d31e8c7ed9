"""ctypes binding of the cache in use (include/rkv.h, "the cache in use"): one
function per C entry point with the same name.

As in ``rkv``: tensor metadata is checked here, outputs the caller did not pass
are allocated, raw pointers and the stream go to the library, and there is no
fallback.  Calls run on the device of their tensors and, unless ``stream`` is
given, on that device's current stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .rkv import (RKV_DTYPE_BF16, RKV_DTYPE_FP32, _PagedDesc, _Q4Cache, _RopeConfig, _RopePlan,
                  _Rows, _check, load)

RKV_MAX_NEW_TOKENS = 64
_DTYPE = {torch.bfloat16: RKV_DTYPE_BF16, torch.float32: RKV_DTYPE_FP32}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
_byref = ctypes.byref


class _Call:
    """The device and stream of a call: entered, its device is current and
    what is allocated belongs to its stream."""

    __slots__ = ("device", "stream", "_dev", "_str")

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError("the tensors must be CUDA tensors")
        self.device, self.stream = t.device, stream
        self._dev = self._str = None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self._dev = torch.cuda.device(self.device)
            self._dev.__enter__()
        if self.stream is not None:
            if self.stream.device != self.device:
                self.__exit__()
                raise ValueError("stream and tensors must be on one device")
            self._str = torch.cuda.stream(self.stream)
            self._str.__enter__()
            return self.stream.cuda_stream
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self._str is not None:
            self._str.__exit__(None, None, None)
            self._str = None
        if self._dev is not None:
            self._dev.__exit__(None, None, None)
            self._dev = None
        return False


def _same_device(ref: torch.Tensor, **tensors):
    dev = ref.device
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")


def _int32(t, name: str, shape):
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)}")


def _dtype(t: torch.Tensor) -> int:
    c = _DTYPE.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")
    return c


def _rows(t: torch.Tensor, name: str, heads, d: int, dtype, tokens: int, per_seq: int) -> _Rows:
    """The rows of [tokens, heads, d] or [seqs, per_seq, heads, d], strides as
    they are."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    sh, st = t.shape, t.stride()
    if t.dim() == 4:
        ok = sh[0] * sh[1] == tokens and sh[1] == per_seq
        seq, tok = st[0], st[1]
    elif t.dim() == 3:
        ok, seq, tok = sh[0] == tokens, per_seq * st[0], st[0]
    else:
        ok, seq, tok = False, 0, 0
    if not ok or sh[-2] != heads or sh[-1] != d:
        raise ValueError(f"{name} must be [{tokens}, {heads}, {d}] or "
                         f"[{tokens // max(per_seq, 1)}, {per_seq}, {heads}, {d}]")
    if st[-1] != 1 and d > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _Rows(t.data_ptr(), seq, tok, st[-2])


def _workspace(ws, name="workspace"):
    if ws is None:
        return None, 0
    if not ws.is_cuda or not ws.is_contiguous() or ws.dtype != torch.uint8:
        raise ValueError(f"{name} must be a contiguous CUDA uint8 tensor")
    if ws.numel() < 256:
        raise ValueError(f"{name} must hold at least 256 bytes")
    return ws.data_ptr(), ws.numel()


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
        self._c = _RopePlan()
        if freqs is not None:
            f = [float(x) for x in freqs]
            if 2 * len(f) != int(rot_dim):
                raise ValueError("freqs must hold rot_dim / 2 angles")
            arr = (ctypes.c_double * max(len(f), 1))(*f)
            rc = load().rkv_rope_init_freqs(int(rot_dim), 1 if interleaved else 0, arr,
                                            float(attn_factor), _byref(self._c))
            _check(rc, "rkv_rope_init_freqs")
        else:
            c = _RopeConfig(int(rot_dim), 1 if interleaved else 0, _SCALING[scaling], float(base),
                            float(factor), float(original_len), float(low), float(high),
                            float(attn_factor))
            _check(load().rkv_rope_init(_byref(c), _byref(self._c)), "rkv_rope_init")

    @property
    def rot_dim(self) -> int:
        return self._c.rot_dim


def rkv_rope_apply(rope: RopePlan, positions, q, k=None, out_q=None, out_k=None,
                   inverse: bool = False, stream=None):
    """q (and k) [tokens, heads, d] or [seqs, n, heads, d] turned by positions
    (int32, one per token); inverse=True turns back, the map of the gradients.
    Outputs may be the inputs.  Returns out_q, or (out_q, out_k) with k."""
    with _Call(q, stream) as s:
        _same_device(q, k=k, positions=positions, out_q=out_q, out_k=out_k)
        if q.dim() not in (3, 4):
            raise ValueError("q must be [tokens, heads, d] or [seqs, n, heads, d]")
        d, hq = q.shape[-1], q.shape[-2]
        per = q.shape[1] if q.dim() == 4 else q.shape[0]
        tokens = q.shape[0] * q.shape[1] if q.dim() == 4 else q.shape[0]
        if positions.dtype != torch.int32 or positions.numel() != tokens \
                or not positions.is_contiguous():
            raise ValueError("positions must be contiguous int32, one per token")
        dt = _dtype(q)
        if out_q is None:
            out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rq = _rows(q, "q", hq, d, q.dtype, tokens, per)
        ro = _rows(out_q, "out_q", hq, d, q.dtype, tokens, per)
        rk = rko = None
        hk = 0
        if k is not None:
            if k.dim() not in (3, 4):
                raise ValueError("k must be [tokens, heads, d] or [seqs, n, heads, d]")
            hk = k.shape[-2]
            if out_k is None:
                out_k = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            rk = _rows(k, "k", hk, d, q.dtype, tokens, per)
            rko = _rows(out_k, "out_k", hk, d, q.dtype, tokens, per)
        elif out_k is not None:
            raise ValueError("out_k without k")
        rc = load().rkv_rope_apply(rope._c, dt, d, tokens, max(per, 1), positions.data_ptr(),
                                   1 if inverse else 0, hq, rq, ro, hk, rk, rko, s)
    _check(rc, "rkv_rope_apply")
    return out_q if k is None else (out_q, out_k)


# ------------------------------------------------------------------ append --

def _append(call, where, cache_args, ref, desc_shape, k, v, block_table, lens, cu_tokens, rope,
            positions, q, out_q, workspace, s):
    nb, H, bs, d = desc_shape
    _same_device(ref, k=k, v=v, block_table=block_table, lens=lens, cu_tokens=cu_tokens,
                 positions=positions, q=q, out_q=out_q, workspace=workspace)
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
    S, mb = block_table.shape
    _int32(block_table, "block_table", (S, mb))
    _int32(lens, "lens", (S,))
    if k.dim() not in (3, 4):
        raise ValueError("k must be [tokens, H, d] or [seqs, n, H, d]")
    tokens = k.shape[0] if k.dim() == 3 else k.shape[0] * k.shape[1]
    if cu_tokens is not None:
        if k.dim() != 3:
            raise ValueError("with cu_tokens, tokens are numbered through: k [tokens, H, d]")
        _int32(cu_tokens, "cu_tokens", (S + 1,))
        per, new = tokens, 0
    else:
        if S == 0 or tokens % S != 0:
            if tokens != 0:
                raise ValueError("without cu_tokens every sequence brings the same number of tokens")
        new = tokens // S if S else 0
        per = new
    if positions is not None and (positions.dtype != torch.int32 or positions.numel() != tokens
                                  or not positions.is_contiguous()):
        raise ValueError("positions must be contiguous int32, one per token")
    if positions is not None and rope is None:
        raise ValueError("positions without a rope")
    dt = _dtype(k)
    rk = _rows(k, "k", H, d, k.dtype, tokens, per)
    rv = _rows(v, "v", H, d, k.dtype, tokens, per)
    rq = ro = None
    G = 1
    if q is not None:
        hq = q.shape[-2]
        if hq % H != 0 or hq == 0:
            raise ValueError("the heads of q must be a multiple of the KV heads")
        G = hq // H
        if out_q is None:
            out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rq = _rows(q, "q", hq, d, k.dtype, tokens, per)
        ro = _rows(out_q, "out_q", hq, d, k.dtype, tokens, per)
    elif out_q is not None:
        raise ValueError("out_q without q")
    wp, _ = _workspace(workspace)
    desc = _PagedDesc(S, H, G, d, bs, nb, mb, dt)
    rc = call(desc, None if rope is None else rope._c, *cache_args, block_table.data_ptr(),
              lens.data_ptr(), tokens, new, None if cu_tokens is None else cu_tokens.data_ptr(),
              None if positions is None else positions.data_ptr(), rk, rv, rq, ro, wp, s)
    _check(rc, where)
    return out_q


def _pool_shape(K_pool, V_pool):
    if K_pool.dim() != 4 or V_pool.shape != K_pool.shape or V_pool.dtype != K_pool.dtype:
        raise ValueError("K_pool, V_pool must be [num_blocks, H, block_size, head_dim] of one dtype")
    if not K_pool.is_contiguous() or not V_pool.is_contiguous():
        raise ValueError("K_pool, V_pool must be contiguous")
    _same_device(K_pool, V_pool=V_pool)
    return K_pool.shape


def rkv_paged_append(K_pool, V_pool, k, v, block_table, lens, cu_tokens=None,
                     rope: RopePlan | None = None, positions=None, q=None, out_q=None,
                     workspace=None, stream=None):
    """Writes the new tokens' keys (turned by rope) and values into a paged
    cache; lens [S] counts the rows with the new tokens.  k, v [tokens, H, d]
    (cu_tokens [S + 1]: sequence s brings tokens cu[s] .. cu[s + 1] - 1;
    without, every sequence the same number) or [S, n, H, d].  positions
    default to the rows written.  q is turned (without a rope: copied) into
    out_q, which is returned (None without q)."""
    with _Call(K_pool, stream) as s:
        shape = _pool_shape(K_pool, V_pool)
        if k.dtype != K_pool.dtype:
            raise ValueError("k, v and the pools must share a dtype")
        return _append(load().rkv_paged_append, "rkv_paged_append",
                       (K_pool.data_ptr(), V_pool.data_ptr()), K_pool, shape, k, v, block_table,
                       lens, cu_tokens, rope, positions, q, out_q, workspace, s)


# ------------------------------------------------------------------ 4 bits --

class Q4Cache:
    """A paged cache held in 4 bits (rkv_q4_cache in include/rkv.h): codes
    uint8 [num_blocks, H, block_size, d / 2], scales bf16 [num_blocks, H,
    block_size, d / 32, 2] (scale, low), for K and for V."""

    def __init__(self, K_codes, K_scales, V_codes, V_scales):
        for t, n in ((K_codes, "K_codes"), (V_codes, "V_codes")):
            if t.dtype != torch.uint8 or t.dim() != 4 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{n} must be contiguous CUDA uint8 [num_blocks, H, block_size, d/2]")
        nb, H, bs, half = K_codes.shape
        for t, n in ((K_scales, "K_scales"), (V_scales, "V_scales")):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != (nb, H, bs, half // 16, 2) \
                    or not t.is_contiguous() or half % 16:
                raise ValueError(f"{n} must be contiguous bf16 [num_blocks, H, block_size, d/32, 2]")
        if V_codes.shape != K_codes.shape:
            raise ValueError("K_codes and V_codes must have one shape")
        _same_device(K_codes, K_scales=K_scales, V_codes=V_codes, V_scales=V_scales)
        self.K_codes, self.K_scales, self.V_codes, self.V_scales = (K_codes, K_scales, V_codes,
                                                                    V_scales)
        self.shape = (nb, H, bs, 2 * half)
        self._c = _Q4Cache(K_codes.data_ptr(), K_scales.data_ptr(), V_codes.data_ptr(),
                           V_scales.data_ptr())


def alloc_q4_cache(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int,
                   device="cuda") -> Q4Cache:
    """A zeroed 4-bit cache (5 bits a value with its scales)."""
    t = []
    for _ in range(2):
        t.append(torch.zeros((num_blocks, num_kv_heads, block_size, head_dim // 2),
                             dtype=torch.uint8, device=device))
        t.append(torch.zeros((num_blocks, num_kv_heads, block_size, head_dim // 32, 2),
                             dtype=torch.bfloat16, device=device))
    return Q4Cache(*t)


def rkv_q4_append(cache: Q4Cache, k, v, block_table, lens, cu_tokens=None,
                  rope: RopePlan | None = None, positions=None, q=None, out_q=None,
                  workspace=None, stream=None):
    """rkv_paged_append into a 4-bit cache (k, v, q bf16 or fp32)."""
    with _Call(cache.K_codes, stream) as s:
        return _append(load().rkv_q4_append, "rkv_q4_append", (cache._c,), cache.K_codes,
                       cache.shape, k, v, block_table, lens, cu_tokens, rope, positions, q, out_q,
                       workspace, s)


def rkv_q4_read(cache: Q4Cache, block_table, lens, n_rows: int, first=None, out_K=None,
                out_V=None, dtype=torch.bfloat16, workspace=None, stream=None):
    """(K, V) rows first[s] .. first[s] + n_rows - 1 of every sequence (first
    None: from row 0) as values [S * H, n_rows, d], the layout of rkv_score and
    rkv_compress.  Rows at or past lens[s] are not written (zeros where the
    output is allocated here)."""
    nb, H, bs, d = cache.shape
    with _Call(cache.K_codes, stream) as s:
        _same_device(cache.K_codes, block_table=block_table, lens=lens, first=first, out_K=out_K,
                     out_V=out_V, workspace=workspace)
        if block_table.dim() != 2:
            raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
        S, mb = block_table.shape
        _int32(block_table, "block_table", (S, mb))
        _int32(lens, "lens", (S,))
        if first is not None:
            _int32(first, "first", (S,))
        shape = (S * H, int(n_rows), d)
        if out_K is None:
            out_K = torch.zeros(shape, dtype=dtype if out_V is None else out_V.dtype,
                                device=cache.K_codes.device)
        if out_V is None:
            out_V = torch.zeros(shape, dtype=out_K.dtype, device=cache.K_codes.device)
        for t, n in ((out_K, "out_K"), (out_V, "out_V")):
            if tuple(t.shape) != shape or not t.is_contiguous() or t.dtype != out_K.dtype:
                raise ValueError(f"{n} must be contiguous {list(shape)}, K and V of one dtype")
        wp, _ = _workspace(workspace)
        desc = _PagedDesc(S, H, 1, d, bs, nb, mb, _dtype(out_K))
        rc = load().rkv_q4_read(desc, cache._c, block_table.data_ptr(), lens.data_ptr(),
                                None if first is None else first.data_ptr(), int(n_rows),
                                out_K.data_ptr(), out_V.data_ptr(), wp, s)
    _check(rc, "rkv_q4_read")
    return out_K, out_V


# --------------------------------------------------------------- attention --

def _attention_shape(q, H: int):
    if q.dim() != 4 or q.shape[2] == 0 or q.shape[2] % H != 0:
        raise ValueError("q must be [num_seqs, n_new, H * gqa_group, d]")
    return q.shape


def rkv_attention_workspace_size(q, num_kv_heads: int, max_rows: int) -> int:
    """Workspace bytes of rkv_paged_attention and rkv_q4_attention for q [S,
    n_new, heads, d] over at most max_rows rows a sequence."""
    S, T, hq, d = _attention_shape(q, num_kv_heads)
    desc = _PagedDesc(S, num_kv_heads, hq // num_kv_heads, d, 1, 1, max(int(max_rows), 1),
                      _dtype(q))
    n = int(load().rkv_attention_workspace_size(_byref(desc), T, int(max_rows)))
    if n == 0:
        raise ValueError("invalid workspace request")
    return n


def alloc_attention_workspace(q, num_kv_heads: int, max_rows: int) -> torch.Tensor:
    """A zero-filled uint8 tensor of rkv_attention_workspace_size() bytes."""
    return torch.zeros(rkv_attention_workspace_size(q, num_kv_heads, max_rows), dtype=torch.uint8,
                       device=q.device)


def _attention(call, where, cache_args, ref, shape, q, block_table, lens, max_rows, scale, out, lse,
               workspace, s):
    nb, H, bs, d = shape
    _same_device(ref, q=q, block_table=block_table, lens=lens, out=out,
                 lse=lse if isinstance(lse, torch.Tensor) else None, workspace=workspace)
    S, T, hq, dq = _attention_shape(q, H)
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks_per_seq]")
    mb = block_table.shape[1]
    _int32(block_table, "block_table", (S, mb))
    _int32(lens, "lens", (S,))
    dt = _dtype(q)
    if max_rows is None:
        max_rows = mb * bs
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, T, hq, d), dtype=q.dtype, device=q.device)
    if lse is True:
        lse = torch.empty((S, T, hq), dtype=torch.float32, device=q.device)
    elif lse is False:
        lse = None
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (S, T, hq)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [num_seqs, n_new, heads]")
    rq = _rows(q, "q", hq, d, q.dtype, S * T, T)
    ro = _rows(out, "out", hq, d, q.dtype, S * T, T)
    desc = _PagedDesc(S, H, hq // H, d, bs, nb, mb, dt)
    if workspace is None:
        n = load().rkv_attention_workspace_size(desc, T, int(max_rows))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    wp, wn = _workspace(workspace)
    rc = call(desc, T, rq, *cache_args, block_table.data_ptr(), lens.data_ptr(), int(max_rows),
              float(scale), ro, None if lse is None else lse.data_ptr(), wp, wn, s)
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
    with _Call(K_pool, stream) as s:
        shape = _pool_shape(K_pool, V_pool)
        if q.dtype != K_pool.dtype:
            raise ValueError("q and the pools must share a dtype")
        return _attention(load().rkv_paged_attention, "rkv_paged_attention",
                          (K_pool.data_ptr(), V_pool.data_ptr()), K_pool, shape, q, block_table,
                          lens, max_rows, scale, out, lse, workspace, s)


def rkv_q4_attention(q, cache: Q4Cache, block_table, lens, max_rows: int | None = None,
                     scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """rkv_paged_attention over a 4-bit cache (q bf16)."""
    with _Call(cache.K_codes, stream) as s:
        return _attention(load().rkv_q4_attention, "rkv_q4_attention", (cache._c,), cache.K_codes,
                          cache.shape, q, block_table, lens, max_rows, scale, out, lse, workspace,
                          s)
