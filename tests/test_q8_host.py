"""Refusals of the 8-bit cache's entry points, answered on the host (no GPU
needed, made-up addresses), and the division by 127 that the append uses."""
import numpy as np

from tests.test_cache_host import BASE, GB, _pdesc, _rows, lib  # noqa: F401


def _cache(ptrs=None):
    from decode_kv_cache_02_gb300 import rkv
    return bytes(rkv._Q8Cache(*(ptrs or [BASE + (8 + i) * GB for i in range(4)])))


def test_q8_append_refusals(lib):  # noqa: F811
    some = object()

    def call(desc=None, cache=some, table=BASE, lens=BASE, n=4, new=1, cu=None, pos=None, k=some,
             v=some, q=None, oq=None, ws=None):
        k = _rows() if k is some else k
        v = _rows(GB) if v is some else v
        cache = _cache() if cache is some else cache
        return lib.rkv_q8_append(desc or _pdesc(), None, cache, table, lens, n, new, cu, pos, k, v, q, oq, ws, None)
    assert call(n=0, new=0) == 0
    assert call(cache=None) == 1
    for i in range(4):
        p = [BASE + (8 + j) * GB for j in range(4)]
        p[i] = 0
        assert call(cache=_cache(p)) == 1
        p[i] = BASE + (8 + i) * GB + 4
        assert call(cache=_cache(p)) == 1
    p = [BASE + (8 + j) * GB for j in range(4)]
    assert call(cache=_cache([p[0], p[0] + 400 * 8 * 16 * 128 - 16, p[2], p[3]])) == 4  # scales inside the codes
    assert call(cache=_cache([p[0], p[1], p[1] + 400 * 8 * 16 * 4 - 16, p[3]])) == 4
    assert call(cache=_cache([BASE, p[1], p[2], p[3]])) == 4                            # the pool is k's memory
    assert call(table=None) == 1 and call(lens=None) == 1
    assert call(n=5) == 1 and call(n=-4, new=-1) == 1
    assert call(k=None) == 1 and call(v=_rows(GB + 8)) == 1
    assert call(oq=_rows(2 * GB)) == 1
    assert call(desc=_pdesc(d=96)) == 2 and call(desc=_pdesc(dtype=2)) == 2
    assert call(desc=_pdesc(bs=24)) != 0
    assert call(ws=BASE + 16) == 3


def test_q8_read_refusals(lib):  # noqa: F811
    def call(desc=None, cache=None, table=BASE, lens=BASE, n=10, k=BASE + 4 * GB, v=BASE + 5 * GB, ws=None):
        return lib.rkv_q8_read(desc or _pdesc(), cache or _cache(), table, lens, None, n, k, v, ws, None)
    assert call(n=0) == 0 and call(n=-1) == 1
    assert call(k=None, v=None) == 1 and call(k=BASE + 8) == 1
    assert call(v=BASE + 4 * GB) == 4
    assert call(k=BASE + 8 * GB) == 4
    assert call(table=None) == 1 and call(lens=None) == 1
    assert call(n=1 << 30) == 2
    assert call(ws=BASE + 16) == 3


def test_q8_attention_refusals(lib):  # noqa: F811
    some = object()

    def call(desc=None, n=1, q=some, cache=some, table=BASE, lens=BASE, rows=100, scale=0.1, out=some, ws=BASE, wb=None):
        desc = desc or _pdesc()
        cache = _cache() if cache is some else cache
        if wb is None:
            wb = max(lib.rkv_attention_workspace_size(desc, n, rows), 256)
        return lib.rkv_q8_attention(desc, n, _rows() if q is some else q, cache, table, lens, rows, scale,
                                    _rows(GB) if out is some else out, None, ws, wb, None)
    assert call(desc=_pdesc(S=0)) == 0
    assert call(desc=_pdesc(dtype=1)) == 2                   # queries are bf16
    assert call(cache=None) == 1
    assert call(n=0) == 1 and call(n=65) == 2
    assert call(rows=0, wb=256) == 1 and call(rows=16 * 80 + 1, wb=1 << 20) == 1
    assert call(scale=float("nan")) == 1
    assert call(ws=None) == 3 and call(wb=0) == 3
    assert call(table=None) == 1 and call(lens=None) == 1
    assert call(out=_rows()) == 4 and call(out=_rows(8 * GB)) == 4
    assert call(q=_rows(8)) == 1


def test_a_127th():
    """x / 127 by the reciprocal and one correction by the remainder: the same bits as the division over a
    binade and at both ends of the range (one multiple-of-997 step through each)."""
    c = np.float32(1) / np.float32(127)
    for e in list(range(0, 12)) + [127, 128, 253, 254]:
        x = ((np.uint32(e) << np.uint32(23)) | np.arange(0, 1 << 23, 997, dtype=np.uint32)).view(np.float32)
        q = x * c
        # fused: the products are exact in 64 bits (x86's or Arm's wider type where there is one)
        w = np.longdouble
        rest = (w(-127) * q.astype(w) + x.astype(w)).astype(np.float32)
        y = (rest.astype(w) * w(c) + q.astype(w)).astype(np.float32)
        assert (y == x / np.float32(127)).all()
