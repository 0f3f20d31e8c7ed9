"""Refusals of the attention over shared prefixes, answered on the host (no GPU
needed, made-up addresses), and its workspace's size."""
import pytest

from tests.test_cache_host import BASE, GB, _pdesc, _rows, lib  # noqa: F401


def _prefixes(table=BASE, lens=BASE, cu=BASE, P=2, mb=40, rows=600):
    from decode_kv_cache_02_gb300 import rkv
    return bytes(rkv._Prefixes(table, lens, cu, P, mb, rows))


def test_prefix_attention_refusals(lib):  # noqa: F811
    some = object()

    def call(desc=None, n=1, q=some, K=BASE + 4 * GB, V=BASE + 6 * GB, pre=some, table=BASE, lens=BASE, rows=100,
             scale=0.1, out=some, lse=None, ws=BASE, wb=None):
        desc = desc or _pdesc()
        pre = _prefixes() if pre is some else pre
        if wb is None:
            wb = max(lib.rkv_prefix_attention_workspace_size(desc, n, rows, pre), 256)
        return lib.rkv_prefix_attention(desc, n, _rows() if q is some else q, K, V, pre, table, lens, rows, scale,
                                        _rows(GB) if out is some else out, lse, ws, wb, None)
    assert call(desc=_pdesc(S=0)) == 0
    assert call(pre=None) == 1
    assert call(pre=_prefixes(P=-1)) == 1
    assert call(pre=_prefixes(mb=0)) == 1 and call(pre=_prefixes(rows=0)) == 1
    assert call(pre=_prefixes(rows=641)) == 1                     # past the prefixes' table
    assert call(pre=_prefixes(mb=1 << 28, rows=(1 << 30) + 1)) == 2
    assert call(pre=_prefixes(cu=None, P=3)) == 1                 # 4 sequences do not divide
    assert call(pre=_prefixes(table=None)) == 1 and call(pre=_prefixes(lens=None)) == 1
    assert call(pre=_prefixes(P=1 << 24)) == 2
    assert call(n=0) == 1 and call(n=65) == 2
    assert call(rows=0, wb=1 << 20) == 1 and call(rows=16 * 80 + 1, wb=1 << 20) == 1
    assert call(scale=float("inf")) == 1
    assert call(ws=None) == 3 and call(ws=BASE + 16) == 3
    assert call(wb=lib.rkv_prefix_attention_workspace_size(_pdesc(), 1, 100, _prefixes()) - 1) == 3
    assert call(table=None) == 1 and call(lens=None) == 1
    assert call(K=None) == 1 and call(V=BASE + 6 * GB + 8) == 1
    assert call(out=_rows()) == 4 and call(out=_rows(4 * GB)) == 4 and call(out=_rows(6 * GB)) == 4
    assert call(q=_rows(8)) == 1 and call(out=_rows(GB, tok=0), n=2) == 1
    assert call(desc=_pdesc(d=96)) == 2 and call(desc=_pdesc(dtype=2)) == 2 and call(desc=_pdesc(G=17)) != 0
    # more units, queries or pool rows than the kernels count
    assert call(pre=_prefixes(P=1 << 20, mb=1 << 26, rows=1 << 30), wb=1 << 40) == 2
    assert call(desc=_pdesc(S=1 << 26, G=16), wb=1 << 60) == 2
    assert call(desc=_pdesc(nb=1 << 26), wb=1 << 40) == 2


@pytest.mark.parametrize("bs", [1, 16, 128])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace(lib, bs, dtype):  # noqa: F811
    """The size does not depend on the blocks or on how the sequences are shared out, covers the own rows' call,
    and is 0 for sizes that are refused."""
    d = _pdesc(S=60, bs=bs, mb=4096 // bs, nb=70000, dtype=dtype)
    size = lib.rkv_prefix_attention_workspace_size
    n = size(d, 1, 1000, _prefixes(P=6, mb=8192 // bs, rows=5000))
    assert n == size(_pdesc(S=60, bs=8, mb=512, nb=70000, dtype=dtype), 1, 1000, _prefixes(P=6, mb=1024, rows=5000, cu=None))
    assert n > lib.rkv_attention_workspace_size(d, 1, 1000) + 60 * 32 * 130 * 4
    assert size(d, 1, 1000, _prefixes(P=0, mb=0, rows=0)) > 0
    assert size(d, 0, 1000, _prefixes()) == 0 and size(d, 1, 1000, None) == 0
    assert size(d, 1, 5000, _prefixes()) == 0
