"""A workspace asked for once, for the largest batch, serves the smaller calls after
it: no GPU needed, sizes and refusals are answered on the host (made-up addresses)."""
import pytest

from tests.test_cache_host import BASE, GB, _pdesc, _rows, lib  # noqa: F401


def least(call):
    """The least workspace that a call takes, by its refusals of smaller ones: with no table, a call whose workspace
    is large enough is refused for the table."""
    low, high = 0, 1 << 32
    assert call(high) == 1
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (mid, high) if call(mid) == 3 else (low, mid)
    return high


def needs(lib, kind, S, G, d, dtype, T, rows):  # noqa: F811
    from decode_kv_cache_02_gb300 import rkv
    desc, q = _pdesc(S=S, H=8, G=G, d=d, dtype=dtype, mb=4096, nb=1 << 20), _rows()
    eight = bytes(rkv._Q8Cache(BASE, BASE + GB, BASE + 2 * GB, BASE + 3 * GB))

    def call(n):
        rest = (None, BASE, rows, 0.1, q, None, BASE, n, None)
        if kind == "paged":
            return lib.rkv_paged_attention(desc, T, q, BASE, BASE, *rest)
        return lib.rkv_q8_attention(desc, T, q, eight, *rest)
    return least(call)


@pytest.mark.parametrize("kind, dtype", [("paged", 0), ("paged", 1), ("q8", 0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 7, 16])
def test_a_workspace_serves_smaller_calls(lib, kind, dtype, d, G):  # noqa: F811
    """What the size is asked for once, for the largest batch, serves every call with fewer sequences, new tokens or
    rows (a decode loop whose sequences end, drafts of other lengths)."""
    def size(S, T, rows):
        return lib.rkv_attention_workspace_size(_pdesc(S=S, H=8, G=G, d=d, dtype=dtype, mb=4096, nb=1 << 20), T, rows)
    tokens = [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 13, 16, 17, 24, 25, 32, 33, 48, 49, 63, 64]
    steps = [(S, T, rows) for S in (1, 2, 5, 16, 70) for T in tokens for rows in (64, 65, 200, 9000)]
    need = {x: needs(lib, kind, x[0], G, d, dtype, *x[1:]) for x in steps}
    got = {x: size(*x) for x in steps}
    for x in steps:
        assert all(got[x] >= max(need[y], got[y]) for y in steps if all(a <= b for a, b in zip(y, x))), x


@pytest.mark.parametrize("bs", [4, 64])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("G, T", [(1, 1), (4, 1), (5, 3), (16, 8)])
def test_a_prefix_workspace_serves_smaller_calls(lib, G, T, dtype, bs):  # noqa: F811
    """The same for prefixes, over the borders of tiles and teams of queries (their choice goes by the sequences a
    prefix) and of the passes (blocks of 4 rows are not the tensor cores')."""
    from decode_kv_cache_02_gb300 import rkv

    def at(S, P, prows):
        return (_pdesc(S=S, H=8, G=G, d=128, dtype=dtype, bs=bs, mb=1 << 14, nb=1 << 20),
                bytes(rkv._Prefixes(BASE, BASE, BASE, P, 1 << 14, prows)))

    def need(S, P, prows):
        desc, pre = at(S, P, prows)
        return least(lambda n: lib.rkv_prefix_attention(desc, T, _rows(), BASE, BASE, pre, None, BASE, 1152, 0.1,
                                                        _rows(GB), None, BASE, n, None))
    steps = [(S, P, rows) for S in (1, 8, 31, 33, 64, 65, 128, 129, 256, 257, 700)
             for P in (0, 1, 2, 9, 100) for rows in (1, 200, 8192)]
    size = {x: lib.rkv_prefix_attention_workspace_size(at(*x)[0], T, 1152, at(*x)[1]) for x in steps}
    low = {x: need(*x) for x in steps}
    for x in steps:
        assert all(size[x] >= max(low[y], size[y]) for y in steps if all(a <= b for a, b in zip(y, x))), x


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_prefix_workspace_serves_fewer_tokens(lib, dtype):  # noqa: F811
    from decode_kv_cache_02_gb300 import rkv
    pre = bytes(rkv._Prefixes(BASE, BASE, BASE, 2, 1 << 14, 5000))
    for S in (1, 7, 40):
        for G in (1, 7, 16):
            desc = _pdesc(S=S, H=8, G=G, d=128, dtype=dtype, mb=1 << 12, nb=1 << 20)
            for rows in (60, 9000):
                size = [lib.rkv_prefix_attention_workspace_size(desc, T, rows, pre) for T in range(1, 65)]
                assert size == sorted(size)
